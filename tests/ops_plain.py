"""Plain 64-bit forms of the operators around the experts, on the CPU, with error bounds for the fp32
arithmetic that the library documents.

A bound counts roundings: a computed quantity is off by at most (number of roundings on its longest
path) * 2^-24 times the same formula taken over magnitudes, then by half a step of the output's type.
"""
import torch

U32 = 2.0 ** -24


def half_step(dtype, ref):
    """Largest rounding error of values `ref` stored in dtype (to nearest; subnormals included)."""
    f = torch.finfo(dtype)
    return ref.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def check(got, ref, bound, what=""):
    """got (any float type) within bound of ref (float64); both finite."""
    g = got.detach().cpu().double()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert torch.isfinite(g).all(), f"{what}: not finite"
    over = (g - ref).abs() - bound
    assert (over <= 0).all(), f"{what}: off by {(g - ref).abs().max():.3g}, {int((over > 0).sum())} values over their bound"


def rounded(got, ref, err, what=""):
    """got = ref computed with absolute error `err`, then rounded to got's type."""
    check(got, ref, err + half_step(got.dtype, ref.abs() + err), what)


# ---- rows by expert ------------------------------------------------------------------------------
def sort_pairs(idx, E):
    """offsets, perm, pos of the stable order by expert (lists of ints walked one by one)."""
    T, k = idx.shape
    flat = idx.reshape(-1).tolist()
    buckets = [[] for _ in range(E)]
    for p, e in enumerate(flat):
        if 0 <= e < E:
            buckets[e].append(p)
    offsets = [0]
    for b in buckets:
        offsets.append(offsets[-1] + len(b))
    order = [p for b in buckets for p in b]
    pos = torch.full((T * k,), -1, dtype=torch.int32)
    for at, p in enumerate(order):
        pos[p] = at
    perm = order + [-1] * (T * k - len(order))
    return (torch.tensor(offsets, dtype=torch.int32), torch.tensor(perm, dtype=torch.int32).reshape(-1),
            pos.view(T, k))


def combine(rows, pos, gates=None, base=None):
    """(out, error bound before rounding) in float64."""
    r, have = rows.double()[pos.clamp(min=0).long()], (pos >= 0).double().unsqueeze(-1)
    g = torch.ones(pos.shape, dtype=torch.float64) if gates is None else torch.where(pos >= 0, gates.double(), 0.0)
    terms = torch.where(have > 0, r, 0.0) * g.unsqueeze(-1)
    out, mag = terms.sum(1), terms.abs().sum(1)
    if base is not None:
        out, mag = out + base.double(), mag + base.double().abs()
    return out, (pos.shape[1] + 1) * U32 * mag


def combine_backward(dout, rows, pos, gates):
    d, r = dout.double(), rows.double()
    drows = torch.zeros(rows.shape, dtype=torch.float64)
    written = torch.zeros(rows.shape[0], dtype=torch.bool)
    dg, mag = torch.zeros(pos.shape, dtype=torch.float64), torch.zeros(pos.shape, dtype=torch.float64)
    for t in range(pos.shape[0]):
        for j in range(pos.shape[1]):
            p = int(pos[t, j])
            if p >= 0:
                drows[p] = gates[t, j].double() * d[t]
                written[p] = True
                dg[t, j] = (d[t] * r[p]).sum()
                mag[t, j] = (d[t] * r[p]).abs().sum()
    # a lane's chain of fused multiply-adds, then five exchanges
    return drows, written, dg, (rows.shape[1] // 32 + 8 + 5) * U32 * mag


# ---- block norms ---------------------------------------------------------------------------------
def chain(H):
    """Roundings on a row sum's longest path: a thread's own values, the warp's five exchanges, the warps."""
    return H // 32 + 32 + 5 + 16


def block_norm(h, y, w_pre, w_post, gate, scale, eps, norm_post):
    """dict of (value, error before rounding) for h, n, r_post, r_pre."""
    f32 = lambda v: torch.tensor(v, dtype=torch.float32).double()  # noqa: E731
    eps, H = f32(eps), h.shape[1]
    out, hh = {}, h.double()
    err = torch.zeros_like(hh)
    rel = (chain(H) / 2 + 4) * U32     # of a row factor: the root halves the sum's error
    if y is not None:
        a = y.double() * f32(scale)
        if gate is not None:
            a = a * gate.double().unsqueeze(1)
        part = 4 * U32
        if norm_post:
            r = 1 / torch.sqrt((y.double() ** 2).mean(1) + eps)
            out["r_post"] = (r, rel * r)
            a, part = a * r.unsqueeze(1), part + rel
        if w_post is not None:
            a = a * w_post.double()
        hh = hh + a
        err = 1.01 * (part * a.abs() + U32 * hh.abs())
        out["h"] = (hh, err)
    r = 1 / torch.sqrt((hh ** 2).mean(1) + eps)
    # the factor moves with h' by at most |error| / |h'| of itself
    rel = rel + err.norm(dim=1) / hh.norm(dim=1).clamp(min=1e-30)
    out["r_pre"] = (r, 1.01 * rel * r)
    n = hh * r.unsqueeze(1)
    ne = err * r.unsqueeze(1) + n.abs() * (rel.unsqueeze(1) + 2 * U32)
    if w_pre is not None:
        n, ne = n * w_pre.double(), ne * w_pre.double().abs()
    out["n"] = (n, 1.01 * ne)
    return out


def block_norm_backward(dn, dh_out, h_out, y, r_pre, r_post, w_pre, w_post, gate, scale):
    """dict of (value, error before rounding), from the row factors as given."""
    T, H = h_out.shape
    zeros = torch.zeros((T, H), dtype=torch.float64)
    dh, mag = (dh_out.double(), dh_out.double().abs()) if dh_out is not None else (zeros, zeros)
    out, c = {}, (chain(H) + 8) * U32
    if dn is not None:
        r = r_pre.double().unsqueeze(1)
        z, u = h_out.double() * r, dn.double() * (1.0 if w_pre is None else w_pre.double())
        dh = dh + r * (u - z * (u * z).mean(1, keepdim=True))
        mag = mag + r * (u.abs() + z.abs() * (u * z).abs().mean(1, keepdim=True))
        out["dw_pre"] = ((dn.double() * z).sum(0), (T + 40) * U32 * (dn.double() * z).abs().sum(0))
    out["dh"] = (dh, c * mag)
    if y is not None:
        s = torch.tensor(scale, dtype=torch.float32).double()
        q = torch.ones((T, 1), dtype=torch.float64) if r_post is None else r_post.double().unsqueeze(1)
        g = torch.ones((T, 1), dtype=torch.float64) if gate is None else gate.double().unsqueeze(1)
        w = torch.ones(H, dtype=torch.float64) if w_post is None else w_post.double()
        x = y.double() * q
        out["dgate"] = (s * (dh * w * x).sum(1), 2 * c * s.abs() * (mag * w.abs() * x.abs()).sum(1))
        out["dw_post"] = ((s * g * dh * x).sum(0), (2 * c + (T + 40) * U32) * (s * g * mag * x).abs().sum(0))
        v, vm = s * g * dh * w, (s * g * w).abs() * mag
        if r_post is None:
            out["dy"] = (v, 2 * c * vm)
        else:
            out["dy"] = (q * (v - x * (v * x).mean(1, keepdim=True)),
                         3 * c * q * (vm + x.abs() * (vm * x.abs()).mean(1, keepdim=True)))
    return out


# ---- microscaled 4-bit floating point ------------------------------------------------------------
MAGNITUDES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def mx4_quantize(v):
    """v [R, K] float64 -> codes [R, K] (0..15), scale codes [R, K/32], by comparing with the midpoints."""
    R, K = v.shape
    b = v.view(R, K // 32, 32)
    bad = ~torch.isfinite(b).all(-1)
    top = torch.where(bad, 1.0, b.abs().amax(-1))
    _, e = torch.frexp(top)                       # top = m 2^e with m in [0.5, 1)
    s = torch.where(top > 0, (e - 1 - 2).clamp(min=-127), -127) + 127
    q = torch.where(bad.unsqueeze(-1), 0.0, b.abs() / torch.exp2((s - 127).double()).unsqueeze(-1))
    code = torch.zeros_like(q, dtype=torch.int64)
    for i in range(7):
        mid = (MAGNITUDES[i] + MAGNITUDES[i + 1]) / 2
        code += ((q > mid) | ((q == mid) & (i % 2 == 1))).long()   # a tie goes to the even code
    code = torch.where(bad.unsqueeze(-1), 0, code + 8 * torch.signbit(b).long())
    return code.view(R, K), torch.where(bad, 255, s)


def mx4_pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8)


def mx4_values(codes, scales):
    """float64 values of packed codes [..., K/2] and scale codes [..., K/32] (NaN for a scale of 255)."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = torch.tensor(MAGNITUDES + [-m for m in MAGNITUDES], dtype=torch.float64)[c]
    unit = torch.where(scales == 255, float("nan"), torch.exp2(scales.double() - 127))
    return v * unit.repeat_interleave(32, dim=-1)


def mx4_product(x, w, offsets):
    """(y, sum of magnitudes) over the segments; rows outside them stay zero."""
    y = torch.zeros((x.shape[0], w.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(y)
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        y[a:b] = x[a:b] @ w[e].t()
        mag[a:b] = x[a:b].abs() @ w[e].abs().t()
    return y, mag
