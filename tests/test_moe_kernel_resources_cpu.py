"""Resource checks on the compiled routing, combine and checkpoint kernels (CPU
only: hipcc emits the gfx950 assembly here): no scratch, no spilled vector
registers, and no kernel that misses the occupancy its launch bounds ask for."""
import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

from block_scaled_precision_token_amd import build
from tests.test_kernel_resources_cpu import _kernel_meta

FILES = {"bsp_route.hip": ["k_route_select", "k_route_place", "k_route_bwd", "k_combine"],
         "bsp_checkpoint.hip": ["k_swiglu_ckpt", "k_swiglu_ckpt_bwd"]}


def assembly(name):
    with tempfile.TemporaryDirectory() as td:
        out = os.path.join(td, "a.s")
        cmd = [build.HIPCC, *build.COMMON, *build.DEVICE, "--cuda-device-only", "-S", os.path.join(build.CSRC, name),
               "-o", out]
        res = subprocess.run(cmd, capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-2000:]
        with open(out) as f:
            return f.read(), res.stderr


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not available")
def test_moe_kernels_use_no_scratch_and_meet_their_occupancy():
    with ThreadPoolExecutor(len(FILES)) as ex:
        built = dict(zip(FILES, ex.map(assembly, FILES)))
    for name, (asm, messages) in built.items():
        assert "occupancy" not in messages, messages
        meta = _kernel_meta(asm)
        for kernel in FILES[name]:
            assert any(kernel in k for k in meta), (kernel, sorted(meta))
        for k, m in meta.items():
            assert m.get("private_segment_fixed_size", 0) == 0, (k, m)
            assert m.get("vgpr_spill_count", 0) == 0, (k, m)
        assert "scratch_" not in asm
