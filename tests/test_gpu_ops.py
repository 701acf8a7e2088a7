"""The operators around the experts against their plain 64-bit forms (tests/ops_plain.py): rows sorted by
expert and back, block norms, microscaled 4-bit floating point, and a run of them together."""
import math
import os
import subprocess
import sys
import threading
import time

import pytest
import torch

import ops_plain as P
from bit_grouped_expert_router_b200 import _lib as M
from bit_grouped_expert_router_b200 import build as B
from bit_grouped_expert_router_b200 import ops

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.build()
    M.lib()


@pytest.fixture(autouse=True)
def _clean_status():
    assert ops.status() == M.MOE_OK
    yield


def gen(*key):
    g = torch.Generator()
    g.manual_seed(sum((i + 1) * 7919 * int(v) for i, v in enumerate(key)) % (1 << 31))
    return g


def draw_idx(g, T, k, E, none=0.0, skew=False):
    e = torch.rand((T, k), generator=g)
    idx = ((e ** 4 if skew else e) * E).long().clamp(max=E - 1).to(torch.int32)
    return torch.where(torch.rand((T, k), generator=g) < none, -1, idx).to(torch.int32)


# ---- rows by expert ------------------------------------------------------------------------------
# one token; the one-launch sort up to 4096 pairs and just over; chunks of several rounds; one expert;
# every pair unrouted; one row of eight values; wide rows in several passes
DISPATCH = [(1, 8, 256, 2048, 0.0), (1, 1, 1, 8, 0.0), (7, 3, 5, 40, 0.3), (128, 32, 256, 64, 0.1), (129, 32, 256, 64, 0.1),
            (4097, 1, 3, 16, 0.0), (700, 6, 200, 136, 0.2), (33, 4, 16, 4104, 0.0), (50, 2, 9, 24, 1.0),
            (9001, 32, 255, 8, 0.05), (512, 8, 1, 72, 0.0)]


@pytest.mark.parametrize("T,k,E,H,none", DISPATCH)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_dispatch(T, k, E, H, none, dtype):
    g = gen(T, k, E, H)
    idx = draw_idx(g, T, k, E, none, skew=T % 2 == 1)
    x = torch.randn((T, H), generator=g).to(dtype)
    rows = torch.full((T * k, H), 7.0, dtype=dtype, device="cuda")
    d = ops.dispatch_rows(x.cuda(), idx.cuda(), E, rows=rows)
    offsets, perm, pos = P.sort_pairs(idx, E)
    assert torch.equal(d.offsets.cpu(), offsets)
    assert torch.equal(d.perm.cpu(), perm)
    assert torch.equal(d.pos.cpu(), pos)
    want = torch.full((T * k, H), 7.0, dtype=dtype)
    kept = int(offsets[E])
    want[:kept] = x[perm[:kept].long() // k]
    assert torch.equal(d.rows.cpu(), want)   # rows behind the last one as they were
    s = ops.dispatch_rows(None, idx.cuda(), E)
    assert s.rows is None
    for a, b in zip(s[1:], d[1:]):
        assert torch.equal(a, b)
    assert ops.status() == M.MOE_OK


def test_dispatch_of_no_tokens():
    d = ops.dispatch_rows(torch.empty((0, 16), device="cuda"), torch.empty((0, 4), dtype=torch.int32, device="cuda"), 5)
    assert d.offsets.tolist() == [0] * 6 and d.rows.shape == (0, 16) and d.pos.shape == (0, 4)
    assert ops.combine_weighted(d.rows, d.pos, torch.empty((0, 4), device="cuda")).shape == (0, 16)


@pytest.mark.parametrize("T", [3, 3000])
def test_dispatch_reports_an_expert_out_of_range_and_drops_it(T):
    idx = draw_idx(gen(T), T, 2, 8)
    idx[1, 1] = 8
    d = ops.dispatch_rows(torch.ones((T, 8), device="cuda"), idx.cuda(), 8)
    assert ops.status() == M.MOE_ERR_DEVICE_BOUNDS
    assert ops.status() == M.MOE_OK
    offsets, perm, pos = P.sort_pairs(idx, 8)
    assert torch.equal(d.offsets.cpu(), offsets) and torch.equal(d.perm.cpu(), perm) and torch.equal(d.pos.cpu(), pos)
    assert int(d.pos[1, 1]) == -1


COMBINE = [(1, 8, 2048), (5, 1, 8), (37, 3, 40), (64, 9, 136), (19, 32, 264), (6, 2, 4104)]


@pytest.mark.parametrize("T,k,H", COMBINE)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_combine_and_the_dispatch_gradient(T, k, H, dtype):
    g = gen(T, k, H)
    _, _, pos = P.sort_pairs(draw_idx(g, T, k, 11, 0.2), 11)
    rows = torch.randn((T * k, H), generator=g).to(dtype)
    used = torch.zeros(T * k, dtype=torch.bool)
    used[pos[pos >= 0].long()] = True
    rows[~used] = float("nan")                       # rows without a pair are not read
    gates = torch.randn((T, k), generator=g)
    gates[pos < 0] = float("nan")                    # nor gates of pairs without a place
    base = torch.randn((T, H), generator=g).to(dtype)
    safe = torch.where(used.unsqueeze(1), rows, torch.zeros((), dtype=dtype))
    for b in (None, base):
        got = ops.combine_weighted(rows.cuda(), pos.cuda(), gates.cuda(), base=None if b is None else b.cuda())
        P.rounded(got, *P.combine(safe, pos, gates, b), "combine")
    P.rounded(ops.dispatch_rows_backward(rows.cuda(), pos.cuda()), *P.combine(safe, pos), "dx")
    into = base.cuda()
    ops.combine_weighted(rows.cuda(), pos.cuda(), gates.cuda(), base=into, out=into)   # in place
    P.rounded(into, *P.combine(safe, pos, gates, base), "in place")
    assert ops.status() == M.MOE_OK


@pytest.mark.parametrize("T,k,H", COMBINE)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_combine_backward(T, k, H, dtype):
    g = gen(T, k, H, 3)
    _, _, pos = P.sort_pairs(draw_idx(g, T, k, 11, 0.2), 11)
    rows = torch.randn((T * k, H), generator=g).to(dtype)
    dout = torch.randn((T, H), generator=g).to(dtype)
    gates = torch.randn((T, k), generator=g)
    drows = torch.full((T * k, H), 5.0, dtype=dtype, device="cuda")
    out, dgates = ops.combine_weighted_backward(dout.cuda(), rows.cuda(), pos.cuda(), gates.cuda(), drows=drows)
    want, written, dg, dg_err = P.combine_backward(dout, rows, pos, gates)
    assert out is drows
    assert (drows.cpu()[~written] == 5.0).all()
    P.rounded(drows.cpu()[written], want[written], want[written].abs() * P.U32, "drows")
    P.check(dgates, dg, dg_err, "dgates")
    mine = rows.cuda()
    ops.combine_weighted_backward(dout.cuda(), mine, pos.cuda(), gates.cuda(), drows=mine)   # in place
    assert torch.equal(mine.cpu()[written], drows.cpu()[written])


def test_gates_gradient_is_the_difference_quotient():
    g = gen(5)
    T, k, H = 6, 3, 32
    _, _, pos = P.sort_pairs(draw_idx(g, T, k, 4), 4)
    rows, dout = torch.randn((T * k, H), generator=g), torch.randn((T, H), generator=g)
    gates = torch.rand((T, k), generator=g)
    _, dgates = ops.combine_weighted_backward(dout.cuda(), rows.cuda(), pos.cuda(), gates.cuda())
    loss = lambda w: float((P.combine(rows, pos, w)[0] * dout.double()).sum())  # noqa: E731
    for t, j in ((0, 0), (3, 2), (5, 1)):
        up, down = gates.double().clone(), gates.double().clone()
        up[t, j] += 0.5
        down[t, j] -= 0.5                            # the loss is linear in the gates: the quotient is exact
        assert abs(loss(up) - loss(down) - float(dgates[t, j])) <= 1e-5 * H


@pytest.mark.parametrize("call", ["combine", "dispatch_backward", "combine_backward", "quantize"])
def test_a_place_out_of_range_is_reported_and_skipped(call):
    T, k, H, n = 5, 2, 32, 10
    pos = torch.arange(n, dtype=torch.int32).view(T, k)
    pos[2, 1] = n
    rows, gates, x = torch.ones((n, H)), torch.ones((T, k)), torch.ones((T, H))
    ok = torch.where(pos < n, pos, -1)
    if call == "combine":
        got = ops.combine_weighted(rows.cuda(), pos.cuda(), gates.cuda())
        assert torch.equal(got.cpu().double(), P.combine(rows, ok)[0])
    elif call == "dispatch_backward":
        got = ops.dispatch_rows_backward(rows.cuda(), pos.cuda())
        assert torch.equal(got.cpu().double(), P.combine(rows, ok)[0])
    elif call == "combine_backward":
        _, dg = ops.combine_weighted_backward(x.cuda(), rows.cuda(), pos.cuda(), gates.cuda())
        assert float(dg[2, 1]) == 0 and float(dg[2, 0]) == H
    else:
        ops.mx4_quantize(x.cuda(), pos=pos.cuda())
    assert ops.status() == M.MOE_ERR_DEVICE_BOUNDS
    assert ops.status() == M.MOE_OK


# ---- block norms ---------------------------------------------------------------------------------
WIDTHS = [8, 64, 256, 264, 1000, 1024, 1032, 2048, 2056, 4096, 5000, 8192, 8200, 16384]
FORMS = {"sandwich": dict(y=True, w_post=True, gate=True, norm_post=True, scale=0.22),
         "add": dict(y=True, w_post=False, gate=False, norm_post=False, scale=1.0),
         "scaled": dict(y=True, w_post=True, gate=False, norm_post=False, scale=-0.7),
         "gated": dict(y=True, w_post=False, gate=True, norm_post=True, scale=2.0),
         "pre": dict(y=False, w_post=False, gate=False, norm_post=False, scale=1.0)}
PAIRS = [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.float32, torch.float32),
         (torch.float32, torch.bfloat16), (torch.float32, torch.float16)]


def norm_inputs(T, H, form, hd, yd):
    f, g = FORMS[form], gen(T, H, len(form))
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(h=(3 * rand(T, H)).to(hd), y=rand(T, H).to(yd) if f["y"] else None, w_pre=1 + 0.1 * rand(H),
                w_post=1 + 0.1 * rand(H) if f["w_post"] else None, gate=torch.rand(T, generator=g) if f["gate"] else None,
                scale=f["scale"], norm_post=f["norm_post"])


def cuda(d):
    return {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in d.items()}


def norm_case(T, H, form, hd, yd):
    a = norm_inputs(T, H, form, hd, yd)
    got = ops.block_norm(**cuda(a), eps=1e-6, out_dtype=yd)
    want = P.block_norm(**a, eps=1e-6)
    for n in ("h", "n", "r_post", "r_pre"):
        if n in want:
            P.rounded(getattr(got, n), *want[n], f"{form} {n}")
        else:
            assert getattr(got, n) is None
    g = gen(T, H, 11)
    h_out = (got.h if got.h is not None else a["h"]).cpu()
    b = dict(dn=torch.randn((T, H), generator=g).to(yd), dh_out=torch.randn((T, H), generator=g).to(hd), h_out=h_out,
             y=a["y"], r_pre=got.r_pre.cpu(), r_post=None if got.r_post is None else got.r_post.cpu(), w_pre=a["w_pre"],
             w_post=a["w_post"], gate=a["gate"], scale=a["scale"])
    for drop in ((), ("dn", "w_pre"), ("dh_out",)):
        c = {n: None if n in drop else v for n, v in b.items()}
        grad, ref = ops.block_norm_backward(**cuda(c)), P.block_norm_backward(**c)
        P.rounded(grad.dh, *ref["dh"], "dh")
        for n, there in (("dw_pre", "dn" not in drop), ("dw_post", a["w_post"] is not None), ("dgate", a["gate"] is not None),
                         ("dy", a["y"] is not None)):
            if there:
                P.rounded(getattr(grad, n), *ref[n], f"{form} {n} without {drop}")
            else:
                assert getattr(grad, n) is None


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("form", FORMS)
def test_block_norm_widths(H, form):
    norm_case(5, H, form, torch.float32, torch.bfloat16)


@pytest.mark.parametrize("hd,yd", PAIRS, ids=str)
@pytest.mark.parametrize("T,H", [(1, 2048), (17, 8), (9, 4096), (3, 16384)])
def test_block_norm_types(T, H, hd, yd):
    norm_case(T, H, "sandwich", hd, yd)


@pytest.mark.parametrize("T,H", [(1500, 48), (6001, 264), (1300, 1200)])
def test_block_norm_backward_over_many_rows(T, H):
    """More rows than the backward pass has blocks (of one or eight rows)."""
    norm_case(T, H, "sandwich", torch.bfloat16, torch.bfloat16)


def test_block_norm_in_place_and_zero_rows():
    a = cuda(norm_inputs(33, 1032, "sandwich", torch.bfloat16, torch.bfloat16))
    want = ops.block_norm(**a)
    h, y = a["h"].clone(), a["y"].clone()
    got = ops.block_norm(h, y, **{n: v for n, v in a.items() if n not in ("h", "y")}, h_out=h, n_out=y)
    assert torch.equal(got.h, want.h) and torch.equal(got.n, want.n) and got.h is h and got.n is y
    zero = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    z = ops.block_norm(zero, zero, norm_post=True, eps=1e-6)
    assert (z.h == 0).all() and (z.n == 0).all()     # mean 0: the factor is 1 / sqrt(eps)
    assert torch.allclose(z.r_pre, torch.full((2,), 1e3, device="cuda"))
    e = ops.block_norm_backward(zero[:0], None, zero[:0], r_pre=z.r_pre[:0], w_pre=torch.ones(64, device="cuda"))
    assert e.dh.shape == (0, 64) and (e.dw_pre == 0).all()


def test_block_norm_gradient_is_the_difference_quotient():
    a = norm_inputs(3, 24, "sandwich", torch.float32, torch.float32)
    g = gen(8)
    dn, dh = torch.randn((3, 24), generator=g), torch.randn((3, 24), generator=g)
    got = ops.block_norm(**cuda(a), eps=1e-6)
    grad = ops.block_norm_backward(dn.cuda(), dh.cuda(), got.h, a["y"].cuda(), r_pre=got.r_pre, r_post=got.r_post,
                                   w_pre=a["w_pre"].cuda(), w_post=a["w_post"].cuda(), gate=a["gate"].cuda(), scale=a["scale"])

    def loss(**change):
        o = P.block_norm(**{**a, **change}, eps=1e-6)
        return float((o["n"][0] * dn.double()).sum() + (o["h"][0] * dh.double()).sum())

    d = 1e-4    # central differences in 64 bits: off by d^2 times third derivatives, here of order one
    for name, of, at in (("h", grad.dh, (1, 5)), ("y", grad.dy, (2, 7)), ("gate", grad.dgate, (1,)),
                         ("w_post", grad.dw_post, (3,)), ("w_pre", grad.dw_pre, (20,))):
        up, down = a[name].double().clone(), a[name].double().clone()
        up[at] += d
        down[at] -= d
        assert abs((loss(**{name: up}) - loss(**{name: down})) / (2 * d) - float(of[at])) < 1e-4, name


# ---- microscaled 4-bit floating point ------------------------------------------------------------
def hard_values(R, K, dtype, seed):
    """Ordinary values, and blocks of zeros, of powers of two and ties, of the type's largest and smallest values."""
    g = gen(R, K, seed)
    v = torch.randn((R, K), generator=g) * torch.exp2(torch.randint(-12, 13, (R, 1), generator=g).float())
    f = torch.finfo(dtype)
    b = v.view(-1, 32)
    n = b.shape[0]
    special = [torch.zeros(32), -torch.zeros(32), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4),
               -torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9] * 4), torch.full((32,), f.max), torch.full((32,), -f.tiny),
               torch.arange(32).float() * f.smallest_normal * f.eps, torch.arange(32) * 2.0 ** -9]
    for i, s in enumerate(special):
        if i < n:
            b[(i * 7) % n] = s
    return v.to(dtype)


@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (130, 96), (65, 2048), (9, 8224), (1000, 512)])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_quantize_bit_for_bit_and_back(R, K, dtype):
    x = hard_values(R, K, dtype, 1)
    codes, scales = ops.mx4_quantize(x.cuda())
    c, s = P.mx4_quantize(x.double())
    assert torch.equal(scales.cpu().long(), s)
    assert torch.equal(codes.cpu(), P.mx4_pack(c))
    values = P.mx4_values(codes.cpu(), scales.cpu())
    for d in (torch.bfloat16, torch.float32):          # exact there
        assert torch.equal(ops.mx4_dequantize(codes, scales, dtype=d).cpu().double(), values)
    half = ops.mx4_dequantize(codes, scales, dtype=torch.float16).cpu()
    assert torch.equal(half, values.to(torch.float32).to(torch.float16))


def test_dequantize_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.uint8).view(16, 16).repeat(16, 1)       # [256, 16]: every pair of codes
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1)
    for d in (torch.bfloat16, torch.float32):
        got = ops.mx4_dequantize(codes.cuda(), scales.cuda(), dtype=d).cpu()
        want = P.mx4_values(codes, scales).to(torch.float32).to(d)                # 6 * 2^127 is an infinity there
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got[~want.isnan()], want[~want.isnan()])


def test_quantize_marks_blocks_that_are_not_finite():
    x = torch.randn((4, 96), generator=gen(2))
    x[0, 3], x[1, 40], x[2, 95] = float("inf"), float("-inf"), float("nan")
    codes, scales = ops.mx4_quantize(x.cuda())
    c, s = P.mx4_quantize(x.double())
    assert torch.equal(scales.cpu().long(), s) and int((s == 255).sum()) == 3
    assert torch.equal(codes.cpu(), P.mx4_pack(c))
    assert torch.equal(ops.mx4_dequantize(codes, scales).isnan().view(4, 3, 32).all(-1).cpu(), s == 255)


@pytest.mark.parametrize("T,k,E,K", [(1, 8, 256, 2048), (50, 3, 7, 96), (20, 9, 4, 8224)])
def test_quantize_into_sorted_rows(T, k, E, K):
    x = torch.randn((T, K), generator=gen(T, K)).to(torch.bfloat16)
    offsets, perm, pos = P.sort_pairs(draw_idx(gen(T), T, k, E, 0.2), E)
    codes = torch.full((T * k, K // 2), 99, dtype=torch.uint8, device="cuda")
    scales = torch.full((T * k, K // 32), 98, dtype=torch.uint8, device="cuda")
    ops.mx4_quantize(x.cuda(), pos=pos.cuda(), codes=codes, scales=scales)
    c, s = P.mx4_quantize(x.double())
    kept = int(offsets[E])
    of = perm[:kept].long() // k
    assert torch.equal(codes.cpu()[:kept], P.mx4_pack(c)[of]) and torch.equal(scales.cpu()[:kept].long(), s[of])
    assert (codes[kept:] == 99).all() and (scales[kept:] == 98).all()


@pytest.mark.parametrize("R,K", [(1, 512), (77, 96), (5, 4128)])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_swiglu_quantize(R, K, dtype):
    x = (2 * torch.randn((R, 2 * K), generator=gen(R, K, 4))).to(dtype)
    codes, scales = ops.mx4_quantize(x.cuda(), act="swiglu")
    gate, up = x.double().chunk(2, dim=1)
    v = gate * torch.sigmoid(gate) * up
    # expf (2 steps), the sum, the quotient, the product: 8 roundings cover the activation in fp32
    d = 8 * P.U32
    _, lo = P.mx4_quantize(v * (1 - d))
    _, hi = P.mx4_quantize(v * (1 + d))
    s = scales.cpu().long()
    assert ((s >= lo) & (s <= hi)).all()
    got = P.mx4_values(codes.cpu(), scales.cpu()).view(R, -1, 32)
    unit = torch.exp2(s.double() - 127).unsqueeze(-1)
    m, gap = v.view(R, -1, 32).abs() / unit, None
    gap = torch.where(m < 2, 0.25, torch.where(m < 4, 0.5, 1.0))       # half the distance of neighbouring values
    gap = torch.where(m > 6, m - 6, gap)
    assert ((got - v.view(R, -1, 32)).abs() <= unit * (gap + m * d)).all()


# one row; segments on both sides of a row tile (224, or 64 where experts average 32 rows or fewer) and of the
# 16-row groups; empty experts; features that end inside a tile; columns that end inside a step (256), an MMA (64) and a scale word
MATMUL = [([1], 8, 32), ([1], 128, 256), ([0, 3, 0, 17], 136, 64), ([224, 225, 0, 16], 256, 512), ([449, 1, 31], 264, 288),
          ([128, 129, 300], 1024, 2048), ([5] * 40, 128, 96), ([700], 72, 1056), ([33, 0, 0, 0], 512, 4128),
          ([2] * 256, 24, 128), ([300] + [0] * 30 + [65], 264, 2080), ([64, 1, 0, 63] + [0] * 20, 128, 5120)]


def matmul_inputs(counts, N, K, extra=0, seed=0):
    g = gen(len(counts), N, K, seed)
    E, R = len(counts), sum(counts) + extra
    offsets = torch.tensor([sum(counts[:e]) for e in range(E + 1)], dtype=torch.int32)
    codes = torch.randint(0, 256, (R, K // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(121, 132, (R, K // 32), generator=g, dtype=torch.uint8)
    w_codes = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    w_scales = torch.randint(118, 126, (E, N, K // 32), generator=g, dtype=torch.uint8)
    return codes, scales, w_codes, w_scales, offsets


@pytest.mark.parametrize("counts,N,K", MATMUL, ids=lambda v: str(v) if isinstance(v, int) else f"{len(v)}x{max(v)}")
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_matmul(counts, N, K, dtype):
    a = matmul_inputs(counts, N, K, extra=3)
    R = a[0].shape[0]
    out = torch.full((R, N), 7.0, dtype=dtype, device="cuda")
    got = ops.mx4_matmul(*[t.cuda() for t in a], out=out)
    assert ops.status() == M.MOE_OK
    y, mag = P.mx4_product(P.mx4_values(a[0], a[1]), P.mx4_values(a[2], a[3]), a[4])
    kept = sum(counts)
    # products of two such values are exact; at most K additions, each off by one step (truncation) of a partial sum
    P.rounded(got[:kept], y[:kept], K * 2.0 ** -23 * mag[:kept], "y")
    assert (got[kept:] == 7.0).all()    # rows behind the last segment as they were


def test_matmul_of_exact_sums_is_exact():
    """Integer operands with unit scales: every partial sum is an integer below 2^24, so fp32 is exact whatever
    the order of the additions."""
    codes, scales, w_codes, w_scales, offsets = matmul_inputs([70, 0, 260], 192, 1024, seed=3)
    keep = torch.tensor([0x00, 0x02, 0x04, 0x05, 0x06, 0x07, 0x0A, 0x0C, 0x0F])   # whole numbers only
    for c in (codes, w_codes):
        lo, hi = keep[c.long() % 9], keep[c.long() // 9 % 9]
        c.copy_((lo | hi << 4).to(torch.uint8))
    scales.fill_(127)
    w_scales.fill_(127)
    got = ops.mx4_matmul(*[t.cuda() for t in (codes, scales, w_codes, w_scales, offsets)], dtype=torch.float32)
    y, _ = P.mx4_product(P.mx4_values(codes, scales), P.mx4_values(w_codes, w_scales), offsets)
    assert torch.equal(got.cpu().double(), y)


def test_matmul_scales_act_on_their_own_block_only():
    """One row and feature at a time: each block of 32 columns times its own two powers of two."""
    K, N, R = 512, 128, 224
    codes, scales = torch.full((R, K // 2), 0x22, dtype=torch.uint8), torch.zeros((R, K // 32), dtype=torch.uint8)
    w_codes, w_scales = torch.full((1, N, K // 2), 0x22, dtype=torch.uint8), torch.full((1, N, K // 32), 127, dtype=torch.uint8)
    for r in range(R):                       # row r: ones in block r % 16 scaled by 2^(r % 7), other blocks zero
        codes[r] = 0
        codes[r, 16 * (r % 16):16 * (r % 16) + 16] = 0x22
        scales[r, r % 16] = 127 + r % 7
    for n in range(N):
        for b in range(K // 32):
            w_scales[0, n, b] = 127 + (n + b) % 5
    offsets = torch.tensor([0, R], dtype=torch.int32)
    got = ops.mx4_matmul(*[t.cuda() for t in (codes, scales, w_codes, w_scales, offsets)], dtype=torch.float32).cpu()
    r, n = torch.arange(R).view(-1, 1), torch.arange(N).view(1, -1)
    assert torch.equal(got, 32.0 * torch.exp2(((r % 7) + (n + r % 16) % 5).float()))


def test_matmul_keeps_not_finite_rows_apart():
    a = list(matmul_inputs([40, 30], 128, 256, seed=7))
    a[1][3, 2] = 255                          # a NaN scale in one row only
    got = ops.mx4_matmul(*[t.cuda() for t in a]).cpu()
    bad = got.isnan().all(1)
    assert bad.nonzero().flatten().tolist() == [3] and torch.isfinite(got[~bad]).all()


def test_matmul_holds_bad_offsets_to_the_rows_and_reports_them():
    a = list(matmul_inputs([20, 30], 64, 128, seed=9))
    a[4] = torch.tensor([-4, 20, 90], dtype=torch.int32)
    got = ops.mx4_matmul(*[t.cuda() for t in a])
    assert ops.status() == M.MOE_ERR_DEVICE_BOUNDS
    y, mag = P.mx4_product(P.mx4_values(a[0], a[1]), P.mx4_values(a[2], a[3]), torch.tensor([0, 20, 50]))
    P.rounded(got, y, 128 * 2.0 ** -23 * mag)
    a[4] = torch.tensor([0, 40, 20], dtype=torch.int32)      # a decreasing pair: an empty segment
    out = torch.full((50, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    got = ops.mx4_matmul(*[t.cuda() for t in a], out=out)
    assert ops.status() == M.MOE_ERR_DEVICE_BOUNDS
    y, mag = P.mx4_product(P.mx4_values(a[0], a[1]), P.mx4_values(a[2], a[3]), torch.tensor([0, 40, 40]))
    P.rounded(got[:40], y[:40], 128 * 2.0 ** -23 * mag[:40])
    assert (got[40:] == 7.0).all()


def test_matmul_keeps_segments_of_unsound_offsets_apart():
    """Offsets that swing up and down: an expert starts at the largest offset so far, so no row has two experts."""
    E = 200
    a = list(matmul_inputs([0] * (E - 1) + [90], 128, 64, seed=11))
    a[4] = torch.tensor([(0, 90, 30, 60)[e % 4] for e in range(E + 1)], dtype=torch.int32)
    got = ops.mx4_matmul(*[t.cuda() for t in a])
    assert ops.status() == M.MOE_ERR_DEVICE_BOUNDS
    y, mag = P.mx4_product(P.mx4_values(a[0], a[1]), P.mx4_values(a[2], a[3]), torch.tensor([0] + [90] * E))
    P.rounded(got, y, 64 * 2.0 ** -23 * mag)


# ---- together ------------------------------------------------------------------------------------
def test_equal_calls_give_equal_bits_on_any_stream():
    g = gen(1)
    idx = draw_idx(g, 300, 4, 16).cuda()
    x = torch.randn((300, 512), generator=g).to(torch.bfloat16).cuda()
    w = [t.cuda() for t in matmul_inputs([1] * 16, 256, 512)[2:4]]
    gates = torch.rand((300, 4), generator=g).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    for stream in (None, s, None, s):
        d = ops.dispatch_rows(x, idx, 16, stream=stream)
        c, sc = ops.mx4_quantize(x, pos=d.pos, stream=stream)
        y = ops.mx4_matmul(c, sc, *w, d.offsets, stream=stream)
        outs.append((d.rows, y, ops.combine_weighted(y, d.pos, gates, stream=stream),
                     *ops.combine_weighted_backward(x[:, :256].contiguous() if stream is None else outs[0][5], y, d.pos, gates,
                                                    stream=stream), x[:, :256].contiguous() if not outs else outs[0][5]))
    torch.cuda.synchronize()
    for o in outs[1:]:
        for p, q in zip(outs[0], o):
            assert torch.equal(p, q)


def test_calls_from_threads_of_their_own():
    """A thread whose first CUDA call is the operator, and several at once on streams of their own."""
    a = [t.cuda() for t in matmul_inputs([70, 30], 128, 256, seed=5)]
    want = ops.mx4_matmul(*a)
    outs = [torch.zeros_like(want) for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=lambda i=i: [ops.mx4_matmul(*a, out=outs[i], stream=streams[i]) for _ in range(5)])
               for i in range(4)]
    one = threading.Thread(target=lambda: ops._ext().mx4_matmul(*a, outs[0], M.MOE_DTYPE_BF16))
    one.start()
    one.join()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and ops.status() == M.MOE_OK


def test_captured_in_a_graph_and_replayed_on_new_inputs():
    g = gen(4)
    T, k, E, H, N = 600, 8, 32, 256, 128       # 4800 pairs: the sort in several launches
    idx, x = draw_idx(g, T, k, E).cuda(), torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    gates, w = torch.rand((T, k), generator=g).cuda(), [t.cuda() for t in matmul_inputs([1] * E, N, H)[2:4]]
    res = torch.randn((T, N), generator=g).to(torch.bfloat16).cuda()
    wn = torch.ones(N, device="cuda")

    def step():
        d = ops.dispatch_rows(x, idx, E)
        c, sc = ops.mx4_quantize(x, pos=d.pos)
        y = ops.mx4_matmul(c, sc, *w, d.offsets)
        o = ops.combine_weighted(y, d.pos, gates)
        n = ops.block_norm(res, o, w_pre=wn)
        b = ops.block_norm_backward(n.n, None, n.h, o, r_pre=n.r_pre, w_pre=wn)
        return (d.rows, d.perm, o, n.h, n.n, b.dh, b.dw_pre, *ops.combine_weighted_backward(b.dy, y, d.pos, gates))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (1, 2):
        idx.copy_(draw_idx(gen(seed), T, k, E, 0.1))
        x.copy_(torch.randn((T, H), generator=gen(seed)).to(torch.bfloat16))
        for t in (held[0], held[7]):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        kept = int((idx >= 0).sum())
        again = step()
        for i, (p, q) in enumerate(zip(held, again)):
            assert torch.equal(p[:kept], q[:kept]) if i in (0, 7) else torch.equal(p, q), i
    assert ops.status() == M.MOE_OK


def test_captured_by_a_process_that_made_no_call_before():
    """The kernels are loaded while the capture runs."""
    code = """
import sys
sys.path[:0] = [%r, %r]
import torch
from bit_grouped_expert_router_b200 import ops
x, idx = torch.randn(700, 64, device="cuda"), torch.zeros(700, 8, dtype=torch.int32, device="cuda")
w, ws = torch.zeros(2, 16, 32, dtype=torch.uint8, device="cuda"), torch.zeros(2, 16, 2, dtype=torch.uint8, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    d = ops.dispatch_rows(x, idx, 2)
    c, s = ops.mx4_quantize(x, pos=d.pos)
    y = ops.mx4_matmul(c, s, w, ws, d.offsets)
    n = ops.block_norm(x, x, norm_post=True, w_post=x[0].clone())
    b = ops.block_norm_backward(n.n, n.h, n.h, x, r_pre=n.r_pre, r_post=n.r_post, w_post=x[0].clone())
g.replay()
torch.cuda.synchronize()
assert ops.status() == 0 and torch.equal(d.rows[5599], x[699]) and (y == 0).all()
print("captured")
""" % (os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


def test_offsets_and_perm_are_those_of_moe_route():
    from bit_grouped_expert_router_b200 import synth
    shape = synth.WORKLOADS["tiny"]
    w = {n: v.cuda() if v is not None else None for n, v in synth.make_layer(shape).items()}
    layer = M.Layer.from_shape(w, shape, max_tokens=shape.T)
    r = layer.route(synth.make_x(shape).cuda())
    d = ops.dispatch_rows(None, r["idx"], shape.E)
    assert torch.equal(d.offsets, r["offsets"]) and torch.equal(d.perm, r["perm"])
    layer.close()


def test_rows_past_32_bit_offsets():
    """Row bytes and elements beyond 2^31: the last rows land where they belong."""
    T, k, H = 4200, 8, 65536                   # 33,600 rows of 128 KiB: 4.4 GB each side
    idx = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    x = torch.arange(T, device="cuda").to(torch.float32).view(T, 1).expand(T, H).to(torch.bfloat16).contiguous()
    d = ops.dispatch_rows(x, idx, 1)
    probe = torch.tensor([0, 1, T * k // 2, T * k - 1], device="cuda")
    assert torch.equal(d.rows[probe], x[probe // k])
    got = ops.dispatch_rows_backward(d.rows, d.pos)
    assert torch.equal(got[-1].float(), 8 * x[-1].float()) and torch.equal(got[T // 2].float(), 8 * x[T // 2].float())
    assert math.prod(d.rows.shape) > 1 << 31


def test_tensors_that_do_not_fit_are_refused():
    x, idx = torch.zeros((4, 64), device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    rows, gates = torch.zeros((8, 64), device="cuda"), torch.zeros((4, 2), device="cuda")
    codes, scales = ops.mx4_quantize(x)
    w, ws, off = codes.view(1, 4, 32), scales.view(1, 4, 2), torch.zeros(2, dtype=torch.int32, device="cuda")
    bad = [lambda: ops.dispatch_rows(x, idx.long(), 4), lambda: ops.dispatch_rows(x[:3], idx, 4),
           lambda: ops.dispatch_rows(x, idx, 0), lambda: ops.dispatch_rows(x.double(), idx, 4),
           lambda: ops.dispatch_rows(x[:, ::2], idx, 4), lambda: ops.dispatch_rows(x, idx.cpu(), 4),
           lambda: ops.dispatch_rows(x.cpu(), idx, 4), lambda: ops.dispatch_rows(x, idx, 4, rows=rows.half()),
           lambda: ops.dispatch_rows(None, idx, 4, rows=rows), lambda: ops.dispatch_rows(x, idx[0], 4),
           lambda: ops.dispatch_rows_backward(rows.t(), idx), lambda: ops.combine_weighted(rows, idx, gates.half()),
           lambda: ops.combine_weighted(rows, idx, gates[:3]), lambda: ops.combine_weighted(rows, idx, gates, base=rows),
           lambda: ops.combine_weighted(rows, idx, gates, out=x.half()), lambda: ops.combine_weighted_backward(rows, rows, idx, gates),
           lambda: ops.block_norm(x, x[:3]), lambda: ops.block_norm(x, x, w_pre=x), lambda: ops.block_norm(x, x, gate=x[0]),
           lambda: ops.block_norm(x, x, out_dtype=torch.bfloat16), lambda: ops.block_norm(x.half(), x),
           lambda: ops.block_norm(x, None, gate=x[:, 0].contiguous()), lambda: ops.block_norm(x, eps=-1.0),
           lambda: ops.block_norm_backward(x, x, x), lambda: ops.block_norm_backward(x, x, x, r_pre=x[0]),
           lambda: ops.block_norm_backward(None, x, x, w_pre=x[0].contiguous()),
           lambda: ops.mx4_quantize(x[:, :40].contiguous()), lambda: ops.mx4_quantize(x, act="swiglu", pos=idx[:2]),
           lambda: ops.mx4_quantize(x, codes=codes[:3], scales=scales[:3]), lambda: ops.mx4_dequantize(codes, scales[:, :1]),
           lambda: ops.mx4_matmul(codes, scales, w[0], ws, off), lambda: ops.mx4_matmul(codes, scales, w, ws, off[:1]),
           lambda: ops.mx4_matmul(codes, scales, w, ws, off, dtype=torch.float16),
           lambda: ops.mx4_matmul(codes, scales, w[:, :3].contiguous(), ws[:, :3].contiguous(), off)]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, M.MoeError)):
            call()
            print("call", i, "was taken")
    with pytest.raises(ValueError, match="not contiguous"):
        ops.dispatch_rows_backward(torch.zeros((64, 64), device="cuda").t(), idx)
    with pytest.raises(M.MoeError) as e:
        ops.block_norm(x, eps=-1.0)
    assert e.value.code == M.MOE_ERR_INVALID_ARG and "eps" in str(e.value)
    assert ops.status() == M.MOE_OK


def test_product_past_32_bit_offsets():
    """Results beyond 2^31 elements: the last rows land where they belong."""
    R, N, K = 270000, 8192, 32
    codes = torch.full((R, K // 2), 0x22, dtype=torch.uint8, device="cuda")          # ones
    scales = (126 + torch.arange(R, device="cuda") % 4).to(torch.uint8).view(R, 1)
    w = torch.full((1, N, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    ws = (126 + torch.arange(N, device="cuda") % 3).to(torch.uint8).view(1, N, 1)
    y = ops.mx4_matmul(codes, scales, w, ws, torch.tensor([0, R], dtype=torch.int32, device="cuda"))
    assert y.numel() > 1 << 31
    rows = torch.tensor([0, 1, R // 2, (1 << 31) // N, R - 2, R - 1], device="cuda")
    want = 32.0 * torch.exp2((rows % 4 - 1).float()).view(-1, 1) * torch.exp2((torch.arange(N, device="cuda") % 3 - 1).float())
    assert torch.equal(y[rows].float(), want)
    assert ops.status() == M.MOE_OK


def test_integers_and_truths_that_do_not_fit_are_refused():
    idx = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    x = torch.ones((2, 64), device="cuda")
    for E in (2 ** 32 + 4, -2 ** 32 + 4):   # 4 in the low 32 bits
        with pytest.raises(ValueError, match="E"):
            ops.dispatch_rows(None, idx, E)
    for name in ("norm_post", "pre"):
        with pytest.raises(ValueError, match=name):
            ops.block_norm(x, y=x.clone(), **{name: torch.ones(2)})


def test_quantize_to_no_places_is_refused():
    """pos [T, 0] has no address: it must not pass for an absent pos, whose rows go to the rows of their own."""
    x = torch.ones((3, 64), device="cuda")
    codes = torch.full((3, 32), 0x99, dtype=torch.uint8, device="cuda")
    scales = torch.full((3, 2), 0x99, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="pos"):
        ops.mx4_quantize(x, pos=torch.zeros((3, 0), dtype=torch.int32, device="cuda"), codes=codes, scales=scales)
    assert (codes == 0x99).all() and (scales == 0x99).all()


def test_an_error_is_told_once_to_one_of_two_callers():
    """Two threads take the status at a time: one of them gets the error, whoever comes first."""
    idx = torch.full((1, 1), 9, dtype=torch.int32, device="cuda")   # no expert of four
    streams = [torch.cuda.Stream() for _ in range(2)]
    start = threading.Barrier(2, timeout=60)
    got = [[], []]

    def take(i):
        for _ in range(100):
            start.wait()
            if i == 0:
                ops.dispatch_rows(None, idx, 4)
                torch.cuda.current_stream().synchronize()
            start.wait()
            got[i].append(ops.status(streams[i]))

    threads = [threading.Thread(target=take, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(sorted(pair) == sorted((M.MOE_OK, M.MOE_ERR_DEVICE_BOUNDS)) for pair in zip(*got))


def test_swiglu_at_the_ends_of_its_range():
    """Blocks of one value each: the gate's tails, and infinities and NaN in either half."""
    inf, nan = math.inf, math.nan
    pairs = [(100.0, 3.0), (-100.0, 3.0), (-88.0, 1.0), (-80.0, 2.0), (1e30, 1e5), (1e30, 1e10), (-inf, 1.0), (inf, 2.0),
             (1.0, inf), (1.0, -inf), (nan, 1.0), (1.0, nan), (0.0, inf), (-0.0, 5.0), (0.0, 0.0)]
    x = torch.tensor([[0.0] * 31 + [g] + [0.0] * 31 + [u] for g, u in pairs])
    codes, scales = ops.mx4_quantize(x.cuda(), act="swiglu")
    got = ops.mx4_dequantize(codes, scales, torch.float32).cpu()[:, 31].tolist()
    for (g, u), y in zip(pairs, got):
        v = g / (1 + math.exp(-g)) * u if -700 < g < 1e300 else (nan if g == -inf else g * u)
        if not abs(v) <= torch.finfo(torch.float32).max:
            assert math.isnan(y), (g, u, y)
        elif abs(v) < 2.0 ** -119:   # the tail: 0, or the value where it is still one of fp32
            assert abs(y) <= 1.5 * abs(v), (g, u, y)
        else:                        # the largest of its block lies in [4, 8) of the scale and goes to 4 or 6
            assert abs(y - v) <= abs(v) / 4, (g, u, y)


@pytest.mark.parametrize("T,k,K", [(1, 1, 32), (37, 3, 544), (300, 9, 96)])
def test_swiglu_quantize_into_sorted_rows(T, k, K):
    """The activation sent to places gives what the activation in order gives there."""
    g = gen(T, k, K, 11)
    x = torch.randn((T, 2 * K), generator=g).bfloat16().cuda()
    d = ops.dispatch_rows(None, draw_idx(g, T, k, 7, 0.2).cuda(), 7)
    codes, scales = ops.mx4_quantize(x, pos=d.pos, act="swiglu")
    c, s = ops.mx4_quantize(x, act="swiglu")
    kept = int(d.offsets[7])
    of = d.perm[:kept].long() // k
    assert torch.equal(codes[:kept], c[of]) and torch.equal(scales[:kept], s[of])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_swiglu_keeps_the_tail_of_a_gate_whose_product_is_ordinary(dtype):
    """silu(gate) far below one, times an up that brings it back: the value must not be lost on the way.  Each row's
    second block is empty but for one value, the largest of its block: it lies in [4, 8) of the scale and goes to 4
    or 6, so the result is within a quarter of it (and the few roundings on its way)."""
    top = torch.finfo(dtype).max
    pairs = [(g, u) for g in (-63.5, -64.0, -64.5, -80.0, -87.0, -87.5, -88.0, -88.5, -89.0, -92.0, -96.0, -100.0, -103.0)
             for u in (1.0, 1e30, 1e36, -3e38) if abs(u) < top]
    x = torch.zeros((len(pairs), 128))
    for i, (g, u) in enumerate(pairs):
        x[i, 63], x[i, 127] = g, u
    x = x.to(dtype)
    codes, scales = ops.mx4_quantize(x.cuda(), act="swiglu")
    got = ops.mx4_dequantize(codes, scales, torch.float32).cpu().double()
    assert (got[:, :63] == 0).all()
    g, u = x[:, 63].double(), x[:, 127].double()
    v = g * torch.exp(g) / (1 + torch.exp(g)) * u
    held = v.abs() >= 2.0 ** -119          # below it the value ends under the smallest scale
    assert int(held.sum()) >= (len(pairs) // 2 if dtype != torch.float16 else 4)
    assert ((got[:, 63] - v).abs() <= v.abs() * (0.25 + 1e-6))[held].all()
    assert (got[:, 63].abs() <= 1.5 * v.abs() + 2.0 ** -128)[~held].all()


def test_a_tensor_given_to_be_written_is_modified_for_autograd():
    """A graph that saved the buffer's values must refuse them, as after any in-place operation."""
    T, k, H = 3, 2, 64
    rand = lambda *s: torch.rand(s, device="cuda")  # noqa: E731
    idx = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    pos = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k)
    codes, scales = ops.mx4_quantize(rand(T, H))
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    w, off = ops.mx4_quantize(rand(16, H)), torch.tensor([0, T], dtype=torch.int32, device="cuda")
    calls = {"rows": (rand(T * k, H), lambda b: ops.dispatch_rows(rand(T, H), idx, 1, rows=b)),
             "dx": (rand(T, H), lambda b: ops.dispatch_rows_backward(rand(T * k, H), pos, out=b)),
             "out": (rand(T, H), lambda b: ops.combine_weighted(rand(T * k, H), pos, rand(T, k), out=b)),
             "drows": (rand(T * k, H), lambda b: ops.combine_weighted_backward(rand(T, H), rand(T * k, H), pos, rand(T, k), drows=b)),
             "h_out": (rand(T, H), lambda b: ops.block_norm(rand(T, H), rand(T, H), h_out=b)),
             "n_out": (rand(T, H), lambda b: ops.block_norm(rand(T, H), n_out=b)),
             "y": (rand(T, 16), lambda b: ops.mx4_matmul(codes, scales, w[0].view(1, 16, -1), w[1].view(1, 16, -1), off, out=b)),
             "codes": (u8(T, H // 2), lambda b: ops.mx4_quantize(rand(T, H), codes=b)),
             "scales": (u8(T, H // 32), lambda b: ops.mx4_quantize(rand(T, H), scales=b))}
    for name, (buffer, call) in calls.items():
        if buffer.is_floating_point():
            leaf = torch.ones_like(buffer, requires_grad=True)
            loss = (leaf * buffer).sum()
            call(buffer)
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                loss.backward()
        else:
            before = buffer._version
            call(buffer)
            assert buffer._version == before + 1, name
    with torch.inference_mode():
        made = torch.zeros((T, H), device="cuda")
    ops.combine_weighted(rand(T * k, H), pos, torch.ones((T, k), device="cuda"), out=made)   # has no version
    assert float(made.min()) > 0
    assert ops.status() == M.MOE_OK


def test_norm_gradients_of_two_widths_from_two_threads():
    """The C entry points hold no lock: two threads may call one kernel, at widths that take different amounts of shared
    memory, at the same time."""
    L, calls = M.lib(), 20000
    start, got, errors = threading.Barrier(2, timeout=60), [0, 0], []

    def run(i, H):
        try:
            g = torch.Generator().manual_seed(H)
            dn, h = (torch.randn((1, H), generator=g).bfloat16().cuda() for _ in range(2))
            r, w, dw, dh = torch.ones(1, device="cuda"), torch.ones(H, device="cuda"), torch.empty(H, device="cuda"), torch.empty_like(h)
            ws = torch.empty(L.moe_block_norm_backward_workspace(1, H), dtype=torch.uint8, device="cuda")
            want = ops.block_norm_backward(dn, None, h, r_pre=r, w_pre=w)
            s = torch.cuda.Stream()
            torch.cuda.synchronize()
            start.wait()
            for _ in range(calls):
                M.check(L.moe_block_norm_backward(dn.data_ptr(), None, h.data_ptr(), M.MOE_DTYPE_BF16, None, M.MOE_DTYPE_BF16, 1, H,
                                                  r.data_ptr(), None, w.data_ptr(), None, 0, None, 1.0, dh.data_ptr(), None,
                                                  dw.data_ptr(), None, None, ws.data_ptr(), ws.numel(), s.cuda_stream))
                got[i] += 1
            s.synchronize()
            assert torch.equal(dh, want.dh) and torch.equal(dw, want.dw_pre)
        except BaseException as e:
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i, H)) for i, H in enumerate((1032, 2048))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    if errors:
        raise errors[0]
    assert got == [calls, calls] and ops.status() == M.MOE_OK


def test_a_call_that_waits_leaves_other_threads_running():
    """A stream about a second behind fills its launch queue: the next call waits for room, and Python's other threads must
    not wait with it."""
    codes, scales = torch.zeros((32, 64), dtype=torch.uint8, device="cuda"), torch.zeros((32, 4), dtype=torch.uint8, device="cuda")
    ops.mx4_dequantize(codes, scales)
    torch.cuda.synchronize()
    gaps, stop = [0.0], threading.Event()

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    other = threading.Thread(target=tick)
    other.start()
    try:
        behind = torch.cuda.Event()
        torch.cuda._sleep(int(2e9))
        behind.record()
        start = time.perf_counter()
        while not behind.query():
            ops.mx4_dequantize(codes, scales)
        took = time.perf_counter() - start
    finally:
        stop.set()
        other.join()
    torch.cuda.synchronize()
    assert max(gaps) < took / 2, f"another thread waited {max(gaps):.3f} of {took:.3f} s"
    assert ops.status() == M.MOE_OK


def test_refusals_from_many_threads():
    """Errors are raised with the interpreter's lock held again, whatever step found them."""
    x, idx = torch.zeros((4, 64), device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    raised = []

    def refuse():
        for _ in range(200):
            for call, error in ((lambda: ops.dispatch_rows(x[:3], idx, 4), ValueError), (lambda: ops.dispatch_rows(x, idx, 257), M.MoeError),
                                (lambda: ops.block_norm(x, eps=-1.0), M.MoeError), (lambda: ops.mx4_quantize(x.cpu()), ValueError)):
                try:
                    call()
                except error as e:
                    raised.append(str(e))

    threads = [threading.Thread(target=refuse) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert len(raised) == 4 * 200 * 4 and ops.status() == M.MOE_OK


def test_an_allocation_that_fails_raises_torchs_error():
    codes = torch.zeros((1 << 15, 2048), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((1 << 15, 128), dtype=torch.uint8, device="cuda")
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (64 << 20)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError, match="out of memory"):     # 512 MiB of values
            ops.mx4_dequantize(codes, scales, dtype=torch.float32)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert ops.mx4_dequantize(codes, scales, dtype=torch.float32).shape == (1 << 15, 4096)
    assert ops.status() == M.MOE_OK


def test_an_error_is_told_once_and_both_callers_come_to_their_end():
    """As above, with what each caller met: an exception in one of them, or a call left out, is a failure."""
    idx = torch.full((1, 1), 9, dtype=torch.int32, device="cuda")   # no expert of four
    streams = [torch.cuda.Stream() for _ in range(2)]
    start, calls = threading.Barrier(2, timeout=60), 100
    got, errors = [[], []], []

    def take(i):
        try:
            for _ in range(calls):
                start.wait()
                if i == 0:
                    ops.dispatch_rows(None, idx, 4)
                    torch.cuda.current_stream().synchronize()
                start.wait()
                got[i].append(ops.status(streams[i]))
        except BaseException as e:
            errors.append(e)
            start.abort()

    threads = [threading.Thread(target=take, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    if errors:
        raise errors[0]
    assert len(got[0]) == len(got[1]) == calls
    assert all(sorted(pair) == sorted((M.MOE_OK, M.MOE_ERR_DEVICE_BOUNDS)) for pair in zip(*got))


@pytest.mark.parametrize("w_scale", [1, 27, 127, 200, 254])
def test_matmul_of_scales_far_from_one_another(w_scale):
    """Scales at the ends of their range whose product is an ordinary number, or ends above or below fp32."""
    N, K = 128, 64
    x = torch.arange(0, 255, 2)
    scales = x.to(torch.uint8).view(-1, 1).repeat(1, K // 32)
    codes = torch.full((len(x), K // 2), 0x22, dtype=torch.uint8)          # ones
    w, ws = torch.full((1, N, K // 2), 0x22, dtype=torch.uint8), torch.full((1, N, K // 32), w_scale, dtype=torch.uint8)
    offsets = torch.tensor([0, len(x)], dtype=torch.int32)
    got = ops.mx4_matmul(*[t.cuda() for t in (codes, scales, w, ws, offsets)], dtype=torch.float32).cpu()
    want = (64.0 * torch.exp2((x + w_scale - 254).double())).float().view(-1, 1).expand(-1, N)
    normal = want >= torch.finfo(torch.float32).smallest_normal
    assert torch.equal(got[normal], want[normal])
    assert (got[~normal] <= torch.finfo(torch.float32).smallest_normal).all() and (got >= 0).all()
