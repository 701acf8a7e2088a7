"""Workloads of the operators around the experts of a mixture-of-experts block: rows sorted by expert and
back (dispatch, weighted combine, their gradients), the norms before and after the block, and experts
in microscaled 4-bit floating point (quantisation and the grouped product).

With ``own`` false, ``run`` computes each operator in plain torch operations (32-bit arithmetic, rounded
once at the end); with ``own`` true it makes the calls a user of the framework makes.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
BLOCK = 32   # elements that share one scale in the microscaled format


# ---- the cases -----------------------------------------------------------------------------------
def listed():
    return [
        # batch-1 decode: one token's eight experts are sorted and its row copied; pure latency
        dict(name="dispatch_token", op="dispatch", T=1, k=8, E=256, H=2048, dtype="bf16", skew=0.0, pad=0),
        # a whole 16384-token prompt in one call, uneven experts, the padded tail of a batch unrouted
        dict(name="dispatch_long", op="dispatch", T=16384, k=8, E=256, H=2048, dtype="bf16", skew=1.2, pad=61),
        # training: the gradient of the token rows of an odd-sized micro-batch
        dict(name="dispatch_grad", op="dispatch_grad", T=4099, k=8, E=256, H=2048, dtype="bf16", skew=1.1, pad=0),
        # decode of a small batch: expert rows weighted and summed onto the shared expert's row
        dict(name="combine_token", op="combine", T=8, k=8, E=256, H=2048, dtype="bf16", skew=0.0, pad=0, base=True),
        # training: gradients of the expert rows and of the gates
        dict(name="combine_grad", op="combine_grad", T=4096, k=8, E=256, H=2048, dtype="bf16", skew=1.1, pad=0),
        # decode: the residual add and the next block's norm for one token
        dict(name="norm_token", op="norm", T=1, H=2048, dtype="bf16", stream="bf16", form="add"),
        # a long prompt through norms on both sides of the block, gated
        dict(name="norm_prompt", op="norm", T=16384, H=2048, dtype="bf16", stream="bf16", form="sandwich"),
        # training with a 32-bit residual stream: all gradients of the same step
        dict(name="norm_grad", op="norm_grad", T=4096, H=2048, dtype="bf16", stream="fp32", form="sandwich"),
        # loading: one layer's down projections brought into the 4-bit format, read back as values
        dict(name="mx4_weights", op="mx4_weights", R=131072, K=512, dtype="bf16"),
        # decode: one token through the gate/up projections of its eight experts; weight bytes bound
        dict(name="mx4_token", op="mx4_up", T=1, k=8, E=256, N=1024, K=2048, dtype="bf16", skew=0.0),
        # a 4096-token chunk through the gate/up projections, uneven experts
        dict(name="mx4_prompt", op="mx4_up", T=4096, k=8, E=256, N=1024, K=2048, dtype="bf16", skew=0.5),
        # the same chunk: SwiGLU, quantisation and the down projections
        dict(name="mx4_down", op="mx4_down", T=4096, k=8, E=256, N=2048, K=512, dtype="bf16", skew=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "norm", "norm_grad",
                     "mx4_weights", "mx4_up", "mx4_up", "mx4_down"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op.startswith("norm"):
        H = 8 * _log(rng, 8, 1024)
        T = _log(rng, 1, max(1, min(16384, 2048 * 16384 // H)))
        stream = rng.choice([dtype, dtype, "fp32"])
        if dtype == "fp32" and op == "norm_grad":
            T = max(1, T // 4)
        elif dtype == "fp32" or stream == "fp32":
            T = max(1, T // 2)
        return dict(op=op, T=T, H=H, dtype=dtype, stream=stream,
                    form=rng.choice(["sandwich", "add", "pre", "scaled"]))
    if op == "mx4_weights":
        K = BLOCK * _log(rng, 1, 128)
        return dict(op=op, R=_log(rng, 1, max(1, 2 ** 25 // K)), K=K, dtype=dtype)
    E = _log(rng, 1, 256)
    k = rng.randint(1, min(E, 12))
    skew = rng.choice([0.0, 0.5, 1.1])
    if op.startswith("mx4"):
        K = BLOCK * _log(rng, 1, 64)
        N = 8 * _log(rng, 4, 256)
        most = max(1, min(4096, 2 ** 22 // k // max(128, N // 4, K // 4)))
        return dict(op=op, T=_log(rng, 1, most), k=k, E=E, N=N, K=K, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    skew=min(skew, 0.5))
    H = 8 * _log(rng, 8, 512)
    size = 4 if dtype == "fp32" else 2
    T = _log(rng, 1, max(1, min(16384, 2 ** 27 * 2 // (size * k * H))))
    case = dict(op=op, T=T, k=k, E=E, H=H, dtype=dtype, skew=skew, pad=rng.choice([0, 0, T // 7]))
    if op == "combine":
        case["base"] = rng.choice([True, False])
    return case


# ---- inputs --------------------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _routing(g, case):
    """Top-k experts of a router with a log-Zipf prior (uniform for skew 0), and their softmax gates."""
    T, E, k = case["T"], case["E"], case["k"]
    ranks = torch.randperm(E, generator=g, device="cuda").float() + 1
    logits = torch.randn((T, E), generator=g, device="cuda") - case["skew"] * ranks.log()
    top, idx = logits.topk(k, dim=1)
    gates = torch.softmax(top, dim=1)
    idx = idx.to(torch.int32)
    if case.get("pad"):
        idx[T - case["pad"]:] = -1
    return idx.contiguous(), gates.contiguous()


def _sorted(idx, E):
    """Stable counting sort of the (token, slot) pairs by expert: offsets, perm, pos."""
    flat = idx.reshape(-1).long()
    n = flat.numel()
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, E)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=idx.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=idx.device)
    offsets[1:] = torch.cumsum(counts[:E], 0).to(torch.int32)
    place = torch.arange(n, device=idx.device)
    perm = torch.where(place < offsets[E], order, -1).to(torch.int32)
    pos = torch.empty(n, dtype=torch.int32, device=idx.device)
    pos[order] = place.to(torch.int32)
    pos = torch.where(valid, pos, -1).view(idx.shape).to(torch.int32)
    return offsets, perm, pos


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    dt = TYPES[case["dtype"]]
    s = dict(case=case)
    if op in ("dispatch", "dispatch_grad", "combine", "combine_grad"):
        T, k, H = case["T"], case["k"], case["H"]
        s["idx"], s["gates"] = _routing(g, case)
        s["offsets"], s["perm"], s["pos"] = _sorted(s["idx"], case["E"])
        if op == "dispatch":
            s["x"] = _normal(g, (T, H), dt)
        else:
            s["rows"] = _normal(g, (T * k, H), dt)
        if op != "dispatch_grad":   # rows that the call leaves as they are hold zeros
            s["buffer"] = torch.zeros((T * k, H), dtype=dt, device="cuda")
        if op == "combine":
            s["base"] = _normal(g, (T, H), dt) if case["base"] else None
        if op == "combine_grad":
            s["dout"] = _normal(g, (T, H), dt)
        return s
    if op in ("norm", "norm_grad"):
        T, H, form, sd = case["T"], case["H"], case["form"], TYPES[case["stream"]]
        s["h"] = _normal(g, (T, H), sd, 3.0)
        s["y"] = _normal(g, (T, H), dt) if form != "pre" else None
        s["w_pre"] = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
        s["w_post"] = 1 + 0.1 * torch.randn(H, generator=g, device="cuda") if form in ("sandwich", "scaled") else None
        s["gate"] = torch.rand(T, generator=g, device="cuda") if form == "sandwich" else None
        s["scale"] = 1.0 if form in ("add", "pre") else 0.22
        s["norm_post"] = form == "sandwich"
        if op == "norm_grad":   # what the forward pass left: the new residual and the row factors
            s["h_out"], _, s["r_post"], s["r_pre"] = _norm(s, sd, dt)
            s["dn"] = _normal(g, (T, H), dt, 0.1)
            s["dh_out"] = _normal(g, (T, H), sd, 0.1)
        return s
    if op == "mx4_weights":
        s["x"] = _normal(g, (case["R"], case["K"]), dt, 0.02)
        return s
    T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
    idx, _ = _routing(g, case)
    s["offsets"], s["perm"], s["pos"] = _sorted(idx, E)
    ends = s["offsets"].tolist()
    s["most"] = max(b - a for a, b in zip(ends, ends[1:]))   # rows of the fullest expert (the plain form pads to it)
    s["w_codes"] = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s["w_scales"] = torch.randint(118, 123, (E, N, K // BLOCK), generator=g, device="cuda", dtype=torch.uint8)
    s["x"] = _normal(g, (T, K) if op == "mx4_up" else (T * k, 2 * K), dt)
    return s


# ---- plain forms ---------------------------------------------------------------------------------
def _taken(rows, pos):
    """rows[pos] in 32 bits, zeros where pos is negative: [T, k, H]."""
    return rows[pos.clamp(min=0).long()].float() * (pos >= 0).unsqueeze(-1)


def _dispatch(s):
    idx, x = s["idx"], s["x"]
    offsets, perm, pos = _sorted(idx, s["case"]["E"])
    kept = (perm >= 0).unsqueeze(1)
    rows = torch.where(kept, x[perm.clamp(min=0).long() // idx.shape[1]], s["buffer"])
    return rows, offsets, perm, pos


def _combine_grad(s):
    pos, gates, dout = s["pos"], s["gates"], s["dout"].float()
    dgates = (_taken(s["rows"], pos) * dout.unsqueeze(1)).sum(-1)
    perm = s["perm"]
    of = perm.clamp(min=0).long()
    drows = dout[of // pos.shape[1]] * gates.reshape(-1)[of].unsqueeze(1)
    return torch.where((perm >= 0).unsqueeze(1), drows.to(s["rows"].dtype), s["buffer"]), dgates


def _norm(s, sd, dt):
    """The new residual, its norm, and the row factors of the two norms (None for one that is not taken)."""
    h = s["h"].float()
    r_post = None
    if s["y"] is not None:
        a = s["y"].float()
        if s["norm_post"]:
            r_post = torch.rsqrt((a * a).mean(-1) + EPS)
            a = a * r_post.unsqueeze(1)
        if s["w_post"] is not None:
            a = a * s["w_post"]
        if s["gate"] is not None:
            a = a * s["gate"].unsqueeze(1)
        h = h + s["scale"] * a
    r_pre = torch.rsqrt((h * h).mean(-1) + EPS)
    n = h * r_pre.unsqueeze(1) * s["w_pre"]
    return h.to(sd), n.to(dt), r_post, r_pre


def _norm_grad(s):
    h, dn, w = s["h_out"].float(), s["dn"].float(), s["w_pre"]
    H = h.shape[1]
    r = s["r_pre"].unsqueeze(1)
    u = dn * w
    dh = s["dh_out"].float() + r * u - h * (r * r * r) * ((u * h).sum(-1, keepdim=True) / H)
    out = dict(dh=dh.to(s["h"].dtype), dw_pre=(dn * h * r).sum(0))
    if s["y"] is not None:
        y = s["y"].float()
        da = s["scale"] * dh
        a = y
        if s["norm_post"]:
            a = a * s["r_post"].unsqueeze(1)
        z = a
        if s["w_post"] is not None:
            z = a * s["w_post"]
        if s["gate"] is not None:
            out["dgate"] = (da * z).sum(-1)
            da = da * s["gate"].unsqueeze(1)
        v = da
        if s["w_post"] is not None:
            out["dw_post"] = (da * a).sum(0)
            v = da * s["w_post"]
        if s["norm_post"]:
            q = s["r_post"].unsqueeze(1)
            v = q * v - y * (q * q * q) * ((v * y).sum(-1, keepdim=True) / H)
        out["dy"] = v.to(s["y"].dtype)
    return out


def _power(code):
    """2^(code - 127) in 32 bits for a scale code in 0..254."""
    return torch.where(code > 0, code << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantized(v):
    """v[..., K] in 32 bits -> the values its microscaled 4-bit form stands for (exact in 32 bits)."""
    b = v.reshape(v.shape[:-1] + (v.shape[-1] // BLOCK, BLOCK))
    _, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    code = (e - 3 + 127).clamp(0, 254)
    code = torch.where(b.abs().amax(-1, keepdim=True) > 0, code, 0).to(torch.int32)
    q = b.abs() * _power(254 - code)
    step = torch.where(q < 2, 0.5, torch.where(q < 4, 1.0, 2.0))
    q = torch.clamp(torch.round(q / step) * step, max=6.0)   # round: ties to the even multiple of the step
    return (torch.copysign(q, b) * _power(code)).reshape(v.shape)


def _decoded(codes, scales):
    """Packed 4-bit codes and scale codes -> values in 32 bits."""
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (-1, BLOCK)).to(torch.int32)
    m, e = c & 1, (c >> 1) & 3
    v = torch.where(e > 0, (1 + 0.5 * m) * (1 << (e - 1).clamp(min=0)), 0.5 * m)
    v = torch.where(c > 7, -v, v) * _power(scales.to(torch.int32)).unsqueeze(-1)
    return v.reshape(codes.shape[:-1] + (-1,))


def _product(s, x):
    """x[R, K] (32-bit values of the sorted rows) times each row's expert matrix, rounded to bf16: a matrix for each
    row where the rows are few, else the experts' rows padded to the fullest one."""
    E, most = s["case"]["E"], s["most"]
    if x.shape[0] <= E:
        e = torch.searchsorted(s["offsets"][1:].long(), torch.arange(x.shape[0], device=x.device), right=True)
        w = _decoded(s["w_codes"][e], s["w_scales"][e])
        return torch.bmm(w, x.unsqueeze(2)).squeeze(2).to(torch.bfloat16)
    start = s["offsets"][:E].long().unsqueeze(1)
    count = s["offsets"][1:].long().unsqueeze(1) - start
    slot = torch.arange(most, device=x.device).unsqueeze(0)
    at = torch.where(slot < count, start + slot, 0)
    y = torch.bmm(x[at], _decoded(s["w_codes"], s["w_scales"]).transpose(1, 2))
    out = torch.empty((x.shape[0], y.shape[2]), dtype=torch.bfloat16, device=x.device)
    where = torch.arange(x.shape[0], device=x.device)
    e = torch.searchsorted(s["offsets"][1:].long(), where, right=True)
    out[:] = y[e, where - s["offsets"].long()[e]]
    return out


def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        from bit_grouped_expert_router_b200 import ops
        if op == "dispatch":
            d = ops.dispatch_rows(s["x"], s["idx"], case["E"], rows=s["buffer"])
            return d.rows, d.offsets, d.perm, d.pos
        if op == "dispatch_grad":
            return ops.dispatch_rows_backward(s["rows"], s["pos"])
        if op == "combine":
            return ops.combine_weighted(s["rows"], s["pos"], s["gates"], base=s["base"])
        if op == "combine_grad":
            return ops.combine_weighted_backward(s["dout"], s["rows"], s["pos"], s["gates"], drows=s["buffer"])
        if op == "norm":
            r = ops.block_norm(s["h"], s["y"], w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"],
                               scale=s["scale"], eps=EPS, norm_post=s["norm_post"], out_dtype=TYPES[case["dtype"]])
            return [r.h, r.n, r.r_post, r.r_pre] if s["y"] is not None else [None, r.n, None, r.r_pre]
        if op == "norm_grad":
            r = ops.block_norm_backward(s["dn"], s["dh_out"], s["h_out"], s["y"], r_pre=s["r_pre"],
                                        r_post=s["r_post"], w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"],
                                        scale=s["scale"])
            return dict(dh=r.dh, dw_pre=r.dw_pre, dgate=r.dgate, dw_post=r.dw_post, dy=r.dy)
        if op == "mx4_weights":
            codes, scales = ops.mx4_quantize(s["x"])
            return ops.mx4_dequantize(codes, scales, dtype=torch.bfloat16)
        if op == "mx4_up":
            codes, scales = ops.mx4_quantize(s["x"], pos=s["pos"])
        else:
            codes, scales = ops.mx4_quantize(s["x"], act="swiglu")
        return ops.mx4_matmul(codes, scales, s["w_codes"], s["w_scales"], s["offsets"])
    if op == "dispatch":
        return _dispatch(s)
    if op == "dispatch_grad":
        return _taken(s["rows"], s["pos"]).sum(1).to(s["rows"].dtype)
    if op == "combine":
        out = (_taken(s["rows"], s["pos"]) * s["gates"].unsqueeze(-1)).sum(1)
        return (out if s["base"] is None else s["base"].float() + out).to(s["rows"].dtype)
    if op == "combine_grad":
        return _combine_grad(s)
    if op == "norm":
        h, n, r_post, r_pre = _norm(s, s["h"].dtype, TYPES[case["dtype"]])
        return [h if s["y"] is not None else None, n, r_post, r_pre]
    if op == "norm_grad":
        return _norm_grad(s)
    if op == "mx4_weights":
        return _quantized(s["x"].float()).to(torch.bfloat16)
    if op == "mx4_up":
        x = _quantized(s["x"].float())[s["perm"].long() // case["k"]]
    else:
        gate, up = s["x"].float().chunk(2, dim=1)
        x = _quantized(gate / (1 + torch.exp(-gate)) * up)
    return _product(s, x)


# ---- what a pass cannot do without ---------------------------------------------------------------
def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op in ("norm", "norm_grad"):
        n, wide = case["T"] * case["H"], 4 if case["stream"] == "fp32" else 2
        has_y = case["form"] != "pre"
        if op == "norm":   # read h and y, write the new residual (with y) and the norm
            return dict(bytes=n * (wide + size + (wide + size if has_y else 0)), flops=12 * n)
        return dict(bytes=n * (size + 3 * wide + (2 * size if has_y else 0)), flops=24 * n)
    if op == "mx4_weights":   # read once, write the codes and scales, read them, write the values
        n = case["R"] * case["K"]
        return dict(bytes=n * (size + 2) + 2 * (n // 2 + n // BLOCK), flops=6 * n)
    T, k, E = case["T"], case["k"], case["E"]
    if op in ("mx4_up", "mx4_down"):
        R, N, K = T * k, case["N"], case["K"]
        used = min(E, R)
        x = T * K * size if op == "mx4_up" else R * 2 * K * size
        return dict(bytes=x + used * N * K * 17 // 32 + R * N * 2 + 4 * R, flops=2 * R * N * K)
    H, P = case["H"], T * k
    R = (T - case["pad"]) * k
    if op == "dispatch":
        return dict(bytes=(T - case["pad"]) * H * size + R * H * size + 12 * P + 4 * (E + 1), flops=0)
    if op == "dispatch_grad":
        return dict(bytes=R * H * size + T * H * size + 4 * P, flops=R * H)
    if op == "combine":
        return dict(bytes=R * H * size + T * H * size * (2 if case["base"] else 1) + 8 * P, flops=2 * R * H)
    return dict(bytes=2 * R * H * size + T * H * size + 12 * P, flops=3 * R * H)


# ---- the definitions in 64 bits ------------------------------------------------------------------
def _grid(v):
    """Microscaled 4-bit values of v in 64 bits, by the nearest of the eight magnitudes."""
    mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)
    b = v.reshape(-1, BLOCK)
    out = torch.empty_like(b)
    for lo in range(0, b.shape[0], 1 << 19):
        p = b[lo:lo + (1 << 19)]
        top = p.abs().amax(1, keepdim=True)
        exp = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
        exp = torch.where(top >= torch.exp2(exp + 1), exp + 1, torch.where(top < torch.exp2(exp), exp - 1, exp))
        unit = torch.exp2(torch.clamp(exp - 2, -127, 127))
        m = p.abs() / unit
        hi = torch.searchsorted(mags, m.contiguous()).clamp(max=7)
        lo_i = (hi - 1).clamp(min=0)
        dl, dh = m - mags[lo_i], mags[hi] - m
        pick = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo_i)
        pick = torch.where(m >= 6, 7, pick)
        out[lo:lo + (1 << 19)] = torch.sign(p) * mags[pick] * unit
    return out.reshape(v.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        x, idx, k = s["x"].double(), s["idx"].reshape(-1).tolist(), case["k"]
        pairs = [p for _, p in sorted((e, p) for p, e in enumerate(idx) if e >= 0)]
        rows = torch.zeros((case["T"] * k, case["H"]), dtype=torch.float64, device="cuda")
        rows[:len(pairs)] = x[torch.tensor(pairs, device="cuda", dtype=torch.long) // k]
        return rows, None, None, None
    if op in ("dispatch_grad", "combine", "combine_grad"):
        pos, rows = s["pos"].long(), s["rows"]
        T, H = pos.shape[0], rows.shape[1]
        have = pos >= 0
        if op == "combine_grad":
            drows = torch.zeros(rows.shape, dtype=torch.float64, device="cuda")
            dgates = torch.zeros(pos.shape, dtype=torch.float64, device="cuda")
            for j in range(pos.shape[1]):
                t = have[:, j].nonzero().squeeze(1)
                d = s["dout"][t].double()
                dgates[t, j] = (d * rows[pos[t, j]].double()).sum(1)
                drows[pos[t, j]] = d * s["gates"][t, j].double().unsqueeze(1)
            return drows, dgates
        out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        if op == "combine" and s["base"] is not None:
            out += s["base"].double()
        for j in range(pos.shape[1]):
            t = have[:, j].nonzero().squeeze(1)
            w = s["gates"][t, j].double().unsqueeze(1) if op == "combine" else 1.0
            out[t] += w * rows[pos[t, j]].double()
        return out
    if op == "norm":
        h = s["h"].double()
        r_post = None
        if s["y"] is not None:
            y = s["y"].double()
            f = torch.full_like(y, s["scale"])
            if s["norm_post"]:
                r_post = 1 / torch.sqrt(y.pow(2).sum(1) / case["H"] + EPS)
                f *= r_post[:, None]
            if s["gate"] is not None:
                f *= s["gate"].double()[:, None]
            if s["w_post"] is not None:
                f *= s["w_post"].double()[None, :]
            h = h + f * y
        r_pre = 1 / torch.sqrt(h.pow(2).sum(1) / case["H"] + EPS)
        return [h if s["y"] is not None else None, h * r_pre[:, None] * s["w_pre"].double()[None, :], r_post, r_pre]
    if op == "norm_grad":
        # the same step as a function of the saved tensors, its pieces differentiated one by one
        h, dn, w = s["h_out"].double(), s["dn"].double(), s["w_pre"].double()
        r = s["r_pre"].double()[:, None]
        along = (dn * w * h).mean(1, keepdim=True)
        dh = s["dh_out"].double() + r * (dn * w - h * r * r * along)
        out = dict(dh=dh, dw_pre=torch.einsum("th,th->h", dn, h * r), dgate=None, dw_post=None, dy=None)
        if s["y"] is None:
            return out
        y = s["y"].double()
        wp = s["w_post"].double() if s["w_post"] is not None else torch.ones(case["H"], dtype=torch.float64, device="cuda")
        q = s["r_post"].double()[:, None] if s["norm_post"] else torch.ones((case["T"], 1), dtype=torch.float64, device="cuda")
        gate = s["gate"].double()[:, None] if s["gate"] is not None else 1.0
        if s["gate"] is not None:
            out["dgate"] = s["scale"] * torch.einsum("th,th->t", dh, y * q * wp)
        if s["w_post"] is not None:
            out["dw_post"] = torch.einsum("th,th->h", s["scale"] * gate * dh, y * q)
        v = s["scale"] * gate * dh * wp * q
        out["dy"] = v - y * q * q * (v * y).mean(1, keepdim=True) if s["norm_post"] else v
        return out
    if op == "mx4_weights":
        return _grid(s["x"].double())
    if op == "mx4_up":
        x = _grid(s["x"].double())[s["perm"].long() // case["k"]]
    else:
        z = s["x"].double()
        K = case["K"]
        x = _grid(z[:, :K] * torch.sigmoid(z[:, :K]) * z[:, K:])
    ends = s["offsets"].tolist()
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    out = torch.empty((x.shape[0], case["N"]), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        if ends[e + 1] > ends[e]:
            c = s["w_codes"][e].long()
            w = torch.empty((case["N"], case["K"]), dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = table[c % 16], table[c // 16]
            w *= torch.exp2(s["w_scales"][e].double() - 127).repeat_interleave(BLOCK, dim=1)
            out[ends[e]:ends[e + 1]] = x[ends[e]:ends[e + 1]] @ w.t()
    return out
