"""Measured cases of the MoE routing, checkpoint and combine operators.

Five operators that a mixture-of-experts training or serving step runs around
the grouped expert GEMMs:

  route        router logits -> the k experts of every token and their softmax
               weights, per-expert counts, the grouped GEMM's row map and the
               load-balance loss
  route_bwd    gradient of the loss and of the weights to the logits
  ckpt         SwiGLU with a weight per row; its input kept in 8 bits (MXFP8)
  ckpt_bwd     SwiGLU's gradient from the 8-bit checkpoint, h recomputed
  combine      the sum of every token's routed rows

`run` computes each in plain torch operations, or through the library where
`own` is set.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
DEV = "cuda"
S8 = 1 + 1 / 32          # MXFP8 bytes per value


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of a serving loop: nothing but latency
        dict(name="route_decode", op="route", T=1, E=128, k=8, shared=0, norm=True, dtype="f32", aux=False, masked=0.0),
        # the Qwen3-30B-A3B-shaped training batch: 8192 tokens, top-8 of 128
        dict(name="route_8192x128", op="route", T=8192, E=128, k=8, shared=0, norm=True, dtype="f32", aux=True,
             masked=0.0),
        # the DeepSeek-V3-shaped layer: 256 experts and a shared one, bf16 logits, a padded batch
        dict(name="route_4096x256_shared", op="route", T=4096, E=256, k=8, shared=1, norm=True, dtype="bf16", aux=True,
             masked=0.1),
        # a long packed batch, odd sizes, weights not renormalised
        dict(name="route_100003x96", op="route", T=100003, E=96, k=6, shared=0, norm=False, dtype="f32", aux=True,
             masked=0.0),
        dict(name="route_bwd_8192x128", op="route_bwd", T=8192, E=128, k=8, shared=0, norm=True, dtype="f32", aux=True,
             masked=0.0),
        # a long padded batch with 256 experts and a shared one
        dict(name="route_bwd_65537x256", op="route_bwd", T=65537, E=256, k=8, shared=1, norm=False, dtype="bf16",
             aux=True, masked=0.1),
        # a short prompt's rows
        dict(name="ckpt_203x768", op="ckpt", R=203, I=768, dtype="bf16", weighted=True, tail=0),
        # the Qwen3-30B-A3B-shaped batch: 8192 tokens x top-8
        dict(name="ckpt_65536x768", op="ckpt", R=65536, I=768, dtype="bf16", weighted=True, tail=0),
        dict(name="ckpt_bwd_65536x768", op="ckpt_bwd", R=65536, I=768, dtype="bf16", weighted=True, tail=0),
        # the DeepSeek-V3-shaped batch: 4096 tokens x (top-8 + shared), the last rows unused (padding tokens)
        dict(name="ckpt_bwd_36864x2048", op="ckpt_bwd", R=36864, I=2048, dtype="bf16", weighted=True, tail=1500),
        # three tokens of a serving loop, weighted here
        dict(name="combine_3x2048", op="combine", T=3, kk=8, H=2048, dtype="bf16", weighted=True, dropped=0.0),
        # the DeepSeek-V3-shaped layer's output, weights already in h
        dict(name="combine_4096x7168", op="combine", T=4096, kk=9, H=7168, dtype="bf16", weighted=False, dropped=0.1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "ckpt", "ckpt_bwd", "combine"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("route", "route_bwd"):
        E = _log_int(rng, 8, 512)
        T = min(_log_int(rng, 1, 131072), (1 << 24) // E)
        return dict(op=op, T=T, E=E, k=min(E, rng.choice([1, 2, 4, 6, 8, 8, 10])), shared=rng.choice([0, 0, 1, 2]),
                    norm=rng.random() < 0.6, dtype=dtype, aux=rng.random() < 0.8, masked=rng.choice([0.0, 0.05, 0.3]))
    if op in ("ckpt", "ckpt_bwd"):
        I = 32 * _log_int(rng, 2, 128)
        R = min(_log_int(rng, 1, 80000), (1 << 25) // I)
        return dict(op=op, R=R, I=I, dtype=dtype, weighted=rng.random() < 0.7,
                    tail=rng.choice([0, 0, 1 + R // 9]) if R > 1 else 0)
    H = 8 * _log_int(rng, 16, 1024)
    kk = rng.randint(1, 10)
    return dict(op=op, T=min(_log_int(rng, 1, 16384), (1 << 27) // (kk * H)), kk=kk, H=H, dtype=dtype,
                weighted=rng.random() < 0.5, dropped=rng.choice([0.0, 0.1]))


def work(case):
    s = SIZE[case["dtype"]]
    op = case["op"]
    if op in ("route", "route_bwd"):
        T, E, kk = case["T"], case["E"], case["k"] + case["shared"]
        if op == "route":   # logits; experts, weights, pos per token; src, row weight per row
            return {"bytes": T * E * s + T * kk * 20 + 12 * (E + 1), "flops": T * E * (5 + 2 * case["k"])}
        return {"bytes": 2 * T * E * s + T * kk * (8 + 4) + 4 * E, "flops": 12 * T * E}
    if op in ("ckpt", "ckpt_bwd"):
        R, I = case["R"], case["I"]
        if op == "ckpt":
            return {"bytes": R * I * (2 * s + 2 + 2 * S8) + 4 * R, "flops": 14 * R * I}
        return {"bytes": R * I * (s + 2 * S8 + 2 * s + 2) + 8 * R, "flops": 20 * R * I}
    T, kk, H = case["T"], case["kk"], case["H"]
    return {"bytes": T * (kk + 1) * H * s + T * kk * (8 if case["weighted"] else 4), "flops": 2 * T * kk * H}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _logits(case, g):
    """N(0, 1) plus ln of a Zipf(1.1) popularity half mixed with a uniform one;
    a padded batch has unroutable entries, one token without any expert, and
    whatever the padding tokens' memory holds."""
    T, E = case["T"], case["E"]
    rank = torch.randperm(E, generator=g, device=DEV) + 1
    pop = rank.float() ** -1.1
    x = _randn(g, T, E) + (0.5 / E + 0.5 * pop / pop.sum()).log()
    mask = None
    if case["masked"]:
        x = torch.where(_rand(g, T, E) < 0.02, -math.inf, x)
        x[T // 2] = -math.inf
        mask = _rand(g, T) >= case["masked"]
        junk = torch.where(_rand(g, T, E) < 0.5, math.nan, math.inf)
        x = torch.where(mask[:, None], x, junk)
    return x.to(DTYPES[case["dtype"]]), mask


def _h13(case, g):
    return (_randn(g, case["R"], 2 * case["I"]) * 1.5).to(DTYPES[case["dtype"]])


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op in ("route", "route_bwd"):
        T, E, kk = case["T"], case["E"], case["k"] + case["shared"]
        G, R = E + case["shared"], T * kk
        st["logits"], st["mask"] = _logits(case, g)
        if op == "route":
            # the buffers that a training or serving loop keeps
            i32, f32 = torch.int32, torch.float32
            new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
            st["out"] = {"experts": new(T, kk, dtype=i32), "weights": new(T, kk, dtype=f32),
                         "counts": new(G + 1, dtype=i32), "group_offsets": new(G + 1, dtype=torch.int64),
                         "src": new(R, dtype=i32), "pos": new(T, kk, dtype=i32), "row_weights": new(R, dtype=f32)}
            if case["aux"]:
                st["out"].update(prob_sum=new(E, dtype=f32), loss=new(1, dtype=f32))
        else:
            fwd = _route(st["logits"], st["mask"], case)
            st["experts"], st["counts"], st["pos"] = fwd["experts"], fwd["counts"], fwd["pos"]
            st["d_row_weights"] = _randn(g, R) * 0.05
            st["d_loss"] = torch.full((1,), 0.01, device=DEV) if case["aux"] else None
        return st
    if op in ("ckpt", "ckpt_bwd"):
        R = case["R"]
        h13 = _h13(case, g)
        st["row_weights"] = _rand(g, R) * 0.3 if case["weighted"] else None
        st["n_rows"] = torch.tensor([R - case["tail"]], device=DEV) if case["tail"] else None
        if case["tail"]:   # the rows past the last routed one are never written
            h13[R - case["tail"]:] = math.nan
        if op == "ckpt":
            st["h13"] = h13
        else:
            codes, scales = _mxfp8(torch.nan_to_num(h13.float()))
            st["ckpt_codes"], st["ckpt_scales"] = codes, scales
            dh = _randn(g, R, case["I"]) * 0.02
            if case["tail"]:
                dh[R - case["tail"]:] = math.nan
            st["dh"] = dh.to(DTYPES[case["dtype"]])
        return st
    T, kk, H = case["T"], case["kk"], case["H"]
    st["y"] = _randn(g, T * kk, H).to(DTYPES[case["dtype"]])
    pos = torch.randperm(T * kk, generator=g, device=DEV).view(T, kk)
    if case["dropped"]:    # padding tokens have no rows
        pos = torch.where(_rand(g, T, 1) < case["dropped"], -1, pos)
    st["pos"] = pos.to(torch.int32)
    st["weights"] = _rand(g, T, kk) * 0.3 if case["weighted"] else None
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _softmax(logits, mask):
    """f32 softmax rows, 0 where there is nothing to route; which tokens are routed."""
    x = logits.float()
    if mask is not None:
        x = torch.where(mask[:, None], x, -math.inf)
    m = x.max(1, keepdim=True).values
    routed = m > -math.inf
    e = torch.where(routed, (x - m).exp(), 0.0)
    z = e.sum(1, keepdim=True)
    return x, torch.where(routed, e / z, 0.0), routed


def _route(logits, mask, case):
    T, E, k, shared = case["T"], case["E"], case["k"], case["shared"]
    kk, G = k + shared, E + shared
    x, p, routed = _softmax(logits, mask)
    order = x.sort(dim=1, descending=True, stable=True).indices[:, :k]
    have = x.gather(1, order) > -math.inf
    w = torch.where(have, p.gather(1, order), 0.0)
    if case["norm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    experts = torch.where(have, order, -1)
    if shared:
        ids = torch.arange(E, G, device=DEV)[None, :].expand(T, shared)
        experts = torch.cat([experts, torch.where(routed, ids, -1)], 1)
        w = torch.cat([w, routed.float().expand(T, shared)], 1)
    flat = torch.where(experts >= 0, experts, G).reshape(-1)
    counts = torch.zeros(G + 1, dtype=torch.int64, device=DEV).scatter_add_(0, flat, torch.ones_like(flat))
    n = routed.sum()
    counts[G] = n
    offsets = torch.zeros(G + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = counts[:G].cumsum(0)
    perm = flat.sort(stable=True).indices
    row = torch.arange(T * kk, device=DEV)
    used = row < offsets[G]
    pos = torch.empty_like(row).scatter_(0, perm, torch.where(used, row, -1))
    out = {"experts": experts.int(), "weights": w, "counts": counts.int(), "group_offsets": offsets,
           "src": torch.where(used, perm // kk, -1).int(), "pos": pos.view(T, kk).int(),
           "row_weights": torch.where(used, w.reshape(-1)[perm], 0.0)}
    if case["aux"]:
        q = p.sum(0)
        nf = n.clamp(min=1).float()
        out["prob_sum"] = q
        out["loss"] = ((counts[:E].float() / nf * (q / nf)).sum() * (E / k)).reshape(1)
    return out


def _route_bwd(st):
    case = st["case"]
    T, E, k, kk = case["T"], case["E"], case["k"], case["k"] + case["shared"]
    x, p, routed = _softmax(st["logits"], st["mask"])
    ex = st["experts"][:, :k].long()
    have = ex >= 0
    at = torch.where(have, ex, 0)
    pos = st["pos"][:, :k].long()
    dw = torch.where(have, st["d_row_weights"][torch.where(have, pos, 0)], 0.0)
    ps = torch.where(have, p.gather(1, at), 0.0)
    if case["norm"]:
        total = ps.sum(1, keepdim=True)
        w = torch.where(total > 0, ps / total, 0.0)
        d = torch.zeros_like(p).scatter_add_(1, at, w * (dw - (w * dw).sum(1, keepdim=True)))
    else:
        d = torch.zeros_like(p).scatter_add_(1, at, ps * dw) - p * (ps * dw).sum(1, keepdim=True)
    if st["d_loss"] is not None:
        n = st["counts"][-1].clamp(min=1).float()
        f = st["counts"][:E].float() / n
        d = d + st["d_loss"] * (E / k) / n * p * (f - (p * f).sum(1, keepdim=True))
    return d.to(st["logits"].dtype)


def _mxfp8(v):
    """MXFP8 of f32 rows: E4M3 codes under the smallest power of two that keeps a block of 32 within 448."""
    b = v.view(v.shape[0], -1, 32)
    bits = b.abs().amax(2).view(torch.int32)
    k = (bits >> 23) - 135 + ((bits & 0x7FFFFF) > 0x600000).int()
    k = torch.where(bits < 0x800000, -127, k.clamp(-127, 119))
    inv = ((127 - k) << 23).view(torch.float32)
    q = (b * inv[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(v.shape), (k + 127).to(torch.uint8)


def _value8(codes, scales):
    q = codes.view(torch.float8_e4m3fn).float().view(codes.shape[0], -1, 32)
    return (q * scales.view(torch.float8_e8m0fnu).float()[:, :, None]).view(codes.shape)


def _used(st, R):
    return None if st["n_rows"] is None else (torch.arange(R, device=DEV) < st["n_rows"])[:, None]


def _weight(st, R):
    return torch.ones(R, 1, device=DEV) if st["row_weights"] is None else st["row_weights"][:, None]


def _ckpt(st):
    case = st["case"]
    R, I = case["R"], case["I"]
    v = st["h13"].float()
    used = _used(st, R)
    if used is not None:
        v = torch.where(used, v, 0.0)
    gate, up = v[:, :I], v[:, I:]
    h = _weight(st, R) * (gate / (1 + (-gate).exp()) * up)
    codes, scales = _mxfp8(v)
    return {"h": h.to(torch.bfloat16), "ckpt_codes": codes.view(torch.float8_e4m3fn), "ckpt_scales": scales}


def _ckpt_bwd(st):
    case = st["case"]
    R, I = case["R"], case["I"]
    v, dh = _value8(st["ckpt_codes"], st["ckpt_scales"]), st["dh"].float()
    used = _used(st, R)
    if used is not None:
        v, dh = torch.where(used, v, 0.0), torch.where(used, dh, 0.0)
    gate, up, w = v[:, :I], v[:, I:], _weight(st, R)
    s = 1 / (1 + (-gate).exp())
    a = gate * s
    da = w * dh
    d = torch.cat([da * up * s * (1 + gate * (1 - s)), da * a], 1)
    out = {"dh13": d.to(st["dh"].dtype), "h": (w * (a * up)).to(torch.bfloat16)}
    if st["row_weights"] is not None:
        out["d_row_weights"] = (dh * (a * up)).sum(1)
    return out


def _combine(st):
    pos = st["pos"].long()
    rows = torch.where((pos >= 0)[:, :, None], st["y"].float()[pos.clamp(min=0)], 0.0)
    if st["weights"] is not None:
        rows = rows * st["weights"][:, :, None]
    return rows.sum(1).to(st["y"].dtype)


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        from block_scaled_precision_token_amd import ops
        if op == "route":
            return ops.moe_route(st["logits"], case["k"], norm=case["norm"], shared=case["shared"],
                                 token_mask=st["mask"], aux=case["aux"], out=st["out"])
        if op == "route_bwd":
            return ops.moe_route_backward(st["logits"], case["k"], st["experts"], st["counts"],
                                          d_weights=st["d_row_weights"], pos=st["pos"], d_loss=st["d_loss"],
                                          norm=case["norm"], shared=case["shared"], token_mask=st["mask"])
        if op == "ckpt":
            r = ops.swiglu_checkpoint(st["h13"], row_weights=st["row_weights"], n_rows=st["n_rows"])
            return {"h": r["h"], "ckpt_codes": r["ckpt_codes"].view(torch.float8_e4m3fn),
                    "ckpt_scales": r["ckpt_scales"]}
        if op == "ckpt_bwd":
            return ops.swiglu_checkpoint_backward(st["dh"], st["ckpt_codes"], st["ckpt_scales"],
                                                  row_weights=st["row_weights"], n_rows=st["n_rows"])
        return ops.moe_combine(st["y"], st["pos"], weights=st["weights"])
    if op == "route":
        return _route(st["logits"], st["mask"], case)
    if op == "route_bwd":
        return _route_bwd(st)
    if op == "ckpt":
        return _ckpt(st)
    if op == "ckpt_bwd":
        return _ckpt_bwd(st)
    return _combine(st)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_probs(st):
    x = st["logits"].double()
    live = torch.ones(x.shape[0], dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"].bool()
    live = live & (x == x).all(1) & (x.amax(1) > -math.inf)
    p = torch.zeros_like(x)
    p[live] = torch.softmax(x[live], dim=1)
    return p, live


def _exact_choice(case, st):
    """Per token the chosen experts as a 0/1 matrix and the weights as a matrix [T, E]."""
    p, live = _exact_probs(st)
    x = st["logits"].double()
    T, E, k = case["T"], case["E"], case["k"]
    left = torch.where(live[:, None], x, torch.full_like(x, -math.inf))
    picks, weights = [], []
    for _ in range(k):
        best = left.amax(1, keepdim=True)
        first = torch.where(left == best, torch.arange(E, device=DEV), E).amin(1, keepdim=True).clamp(max=E - 1)
        ok = best > -math.inf
        picks.append(torch.where(ok, first, -1))
        weights.append(torch.where(ok, p.gather(1, first), torch.zeros_like(best)))
        left = left.scatter(1, first, -math.inf)
    return p, live, torch.cat(picks, 1), torch.cat(weights, 1)


def _exact_route(case, st):
    p, live, picks, w = _exact_choice(case, st)
    E, k = case["E"], case["k"]
    if case["norm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    rows_w, rows_g = [w], [picks]
    for s in range(case["shared"]):
        rows_w.append(live.double()[:, None])
        rows_g.append(torch.where(live, E + s, -1)[:, None])
    w, groups = torch.cat(rows_w, 1), torch.cat(rows_g, 1)
    row_weights = torch.zeros(w.numel(), dtype=torch.float64, device=DEV)
    at, load = 0, []
    for e in range(E + case["shared"]):       # group by group, tokens in order
        here = w[groups == e]
        row_weights[at:at + here.numel()] = here
        at += here.numel()
        load.append(here.numel())
    out = {"experts": None, "weights": w, "counts": None, "group_offsets": None, "src": None, "pos": None,
           "row_weights": row_weights}
    if case["aux"]:
        n = max(int(live.sum()), 1)
        f = torch.tensor(load[:E], dtype=torch.float64, device=DEV) / (k * n)
        out["prob_sum"] = p.sum(0)
        out["loss"] = (E * (f * p.mean(0) * (p.shape[0] / n)).sum()).reshape(1)
    return out


def _exact_route_bwd(case, st):
    """By automatic differentiation of loss and weights in 64 bits."""
    p, live, picks, _ = _exact_choice(case, st)
    E, k, T = case["E"], case["k"], case["T"]
    x = st["logits"].double()[live].clone().requires_grad_(True)
    q = torch.softmax(x, dim=1)
    sel = picks[live]
    ok = sel >= 0
    w = q.gather(1, sel.clamp(min=0)) * ok
    if case["norm"]:
        w = w / w.sum(1, keepdim=True)
    rows = st["pos"][live][:, :k].long().clamp(min=0)
    total = (w * st["d_row_weights"].double()[rows] * ok).sum()
    if case["aux"]:
        n = max(int(live.sum()), 1)
        load = torch.stack([(sel == e).sum() for e in range(E)]).double()
        total = total + float(st["d_loss"].double()) * E * (load / (k * n) * (q.sum(0) / n)).sum()
    grad = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    if x.numel():
        total.backward()
        grad[live] = x.grad
    return grad


def _pow2(e):
    """2^e as a 64-bit float, e between -1022 and 1023."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_swiglu(gate, up):
    return gate * torch.sigmoid(gate) * up


def _exact_ckpt(case, st):
    R, I, n = case["R"], case["I"], case["R"] - case["tail"]
    v = torch.zeros(R, 2 * I, dtype=torch.float64, device=DEV)
    v[:n] = st["h13"][:n].double()
    w = torch.ones(R, 1, dtype=torch.float64, device=DEV) if st["row_weights"] is None else \
        st["row_weights"].double()[:, None]
    h = _exact_swiglu(v[:, :I], v[:, I:]) * w
    # the E4M3 value nearest to v / 2^k, ties to even, for the smallest k with the block within 448 * 2^k
    blocks = v.view(R, -1, 32)
    top = blocks.abs().amax(2, keepdim=True)
    mant, ex = torch.frexp(top)
    k = torch.where(top > 0, ex - 9 + (mant > 0.875).int(), -127).clamp(-127, 119)
    y = blocks * _pow2(-k)
    _, ey = torch.frexp(y)
    step = _pow2(ey.clamp(min=-5) - 4)
    q = ((y / step).round() * step).clamp(-448, 448)
    return {"h": h, "ckpt_codes": q.view(R, 2 * I), "ckpt_scales": None}


def _exact_ckpt_bwd(case, st):
    R, I, n = case["R"], case["I"], case["R"] - case["tail"]
    code = st["ckpt_codes"].view(torch.float8_e4m3fn).double()
    v = code * _pow2(st["ckpt_scales"].int() - 127).repeat_interleave(32, dim=1)
    gate, up = v[:n, :I], v[:n, I:]
    w = torch.ones(n, 1, dtype=torch.float64, device=DEV) if st["row_weights"] is None else \
        st["row_weights"].double()[:n, None]
    dh = st["dh"][:n].double()
    sig = torch.sigmoid(gate)
    full = lambda m, cols: torch.cat([m, torch.zeros(R - n, cols, dtype=torch.float64, device=DEV)])  # noqa: E731
    dgate = w * dh * up * (sig + gate * sig * (1 - sig))
    dup = w * dh * gate * sig
    out = {"dh13": full(torch.cat([dgate, dup], 1), 2 * I), "h": full(w * _exact_swiglu(gate, up), I)}
    if st["row_weights"] is not None:
        out["d_row_weights"] = full((dh * _exact_swiglu(gate, up)).sum(1, keepdim=True), 1).reshape(-1)
    return out


def _exact_combine(case, st):
    out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=DEV)
    for j in range(case["kk"]):
        at = st["pos"][:, j].long()
        rows = st["y"][at.clamp(min=0)].double() * (at >= 0)[:, None]
        out += rows if st["weights"] is None else rows * st["weights"][:, j:j + 1].double()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _exact_route, "route_bwd": _exact_route_bwd, "ckpt": _exact_ckpt, "ckpt_bwd": _exact_ckpt_bwd,
            "combine": _exact_combine}[case["op"]](case, st)
