"""The block norms over many rows against their 64-bit forms (tests/ops_plain.py, run on the device): every geometry of
the forward pass that large inputs take, and a gradient whose groups of warps walk more rows than their ring has
stages, or several rows without a ring."""
import pytest
import torch

import ops_plain as P
from bit_grouped_expert_router_b200 import _lib as M
from bit_grouped_expert_router_b200 import build as B
from bit_grouped_expert_router_b200 import ops

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
CODE = {BF16: M.MOE_DTYPE_BF16, FP16: M.MOE_DTYPE_FP16, FP32: M.MOE_DTYPE_FP32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.build()
    M.lib()


def plain(f, **a):
    """f's 64-bit form computed on the device, its results brought back."""
    with torch.device("cuda"):
        out = f(**a)
    return {n: tuple(t.cpu() for t in v) for n, v in out.items()}


def inputs(T, H, hd, yd, seed=0):
    g = torch.Generator(device="cuda").manual_seed(T * 7919 + H + seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return dict(h=(3 * rand(T, H)).to(hd), y=rand(T, H).to(yd), w_pre=1 + 0.1 * rand(H), w_post=1 + 0.1 * rand(H),
                gate=torch.rand(T, generator=g, device="cuda"), scale=0.22, norm_post=True), \
        dict(dn=rand(T, H).to(yd), dh_out=rand(T, H).to(hd))


# T, H, types of the stream and of the block, and the rows that a group of warps walks / stages of its ring.  148 blocks,
# or one per row; groups per block and stages by the shared memory that a row's pieces take.
MANY = [(14500, 200, BF16, BF16),    # 16 groups of one warp: 7 rows, 4 stages
        (14500, 264, FP32, FP16),    # the same, two pieces a thread
        (7200, 1000, FP16, FP16),    # 8 groups of two warps: 7 rows, 3 stages
        (3000, 2048, BF16, BF16),    # 4 groups of four warps: 6 rows, 3 stages
        (4096, 2048, FP32, BF16),    # 4 groups: 7 rows, 2 stages
        (1500, 4096, BF16, BF16),    # 2 groups of eight warps: 6 rows, 2 stages
        (740, 4096, FP32, FP32),     # 1 group: 5 rows, 2 stages
        (600, 8192, BF16, BF16),     # 1 group of sixteen warps: 5 rows, 2 stages
        (450, 8192, FP32, BF16),     # no ring: 4 rows
        (450, 8200, FP32, FP16),     # sums in shared memory, no ring: 4 rows
        (450, 16384, BF16, BF16)]    # the same, both pieces of every thread


@pytest.mark.parametrize("T,H,hd,yd", MANY, ids=str)
def test_norm_and_gradient_over_many_rows(T, H, hd, yd):
    a, d = inputs(T, H, hd, yd)
    got = ops.block_norm(**a, eps=1e-6)
    want = plain(P.block_norm, **a, eps=1e-6)
    for n in ("h", "n", "r_post", "r_pre"):
        P.rounded(getattr(got, n), *want[n], n)
    b = dict(**d, h_out=got.h, y=a["y"], r_pre=got.r_pre, r_post=got.r_post, w_pre=a["w_pre"], w_post=a["w_post"],
             gate=a["gate"], scale=a["scale"])
    grad, want = ops.block_norm_backward(**b), plain(P.block_norm_backward, **b)
    for n in ("dh", "dy", "dw_pre", "dw_post", "dgate"):
        P.rounded(getattr(grad, n), *want[n], n)
    again = ops.block_norm_backward(**b)
    for n in ("dh", "dy", "dw_pre", "dw_post", "dgate"):
        assert torch.equal(getattr(grad, n), getattr(again, n)), n     # sums in a fixed order
    assert ops.status() == M.MOE_OK


@pytest.mark.parametrize("T,H,dtype", [(14500, 264, BF16), (7200, 1000, FP32), (2100, 8, FP16), (600, 8192, BF16), (450, 16384, BF16)], ids=str)
def test_norm_alone_over_many_rows(T, H, dtype):
    """Without a block's output: the ring holds two of its four rows, and nothing but dh and dw_pre is left."""
    a, d = inputs(T, H, dtype, dtype, 1)
    x = dict(h=a["h"], w_pre=a["w_pre"])
    none = dict(y=None, w_post=None, gate=None, scale=1.0)
    got = ops.block_norm(**x, eps=1e-6)
    want = plain(P.block_norm, **x, **none, eps=1e-6, norm_post=False)
    assert got.h is None and got.r_post is None
    P.rounded(got.n, *want["n"], "n")
    for dh_out in (None, d["dh_out"]):
        b = dict(dn=d["dn"], dh_out=dh_out, h_out=a["h"], r_pre=got.r_pre, w_pre=a["w_pre"])
        grad, want = ops.block_norm_backward(**b), plain(P.block_norm_backward, **b, **none, r_post=None)
        P.rounded(grad.dh, *want["dh"], "dh")
        P.rounded(grad.dw_pre, *want["dw_pre"], "dw_pre")
        assert grad.dy is None and grad.dw_post is None and grad.dgate is None


@pytest.mark.parametrize("T,H,hd,yd", [(14500, 264, BF16, BF16), (3000, 2048, FP32, BF16), (450, 8192, FP32, FP32), (450, 16384, BF16, BF16)],
                         ids=str)
def test_gradients_written_over_those_they_come_from(T, H, hd, yd):
    """The C entry point: dh may be dh_out and dy may be dn; rows that are read ahead are never rows already written."""
    a, d = inputs(T, H, hd, yd, 2)
    f = ops.block_norm(**a, eps=1e-6)
    want = ops.block_norm_backward(**d, h_out=f.h, y=a["y"], r_pre=f.r_pre, r_post=f.r_post, w_pre=a["w_pre"],
                                   w_post=a["w_post"], gate=a["gate"], scale=a["scale"])
    L = M.lib()
    ws = torch.empty(L.moe_block_norm_backward_workspace(T, H), dtype=torch.uint8, device="cuda")
    dw_pre, dw_post, dgate = (torch.empty(n, device="cuda") for n in (H, H, T))
    dn, dh = d["dn"].clone(), d["dh_out"].clone()
    p = lambda t: t.data_ptr()  # noqa: E731
    M.check(L.moe_block_norm_backward(p(dn), p(dh), p(f.h), CODE[hd], p(a["y"]), CODE[yd], T, H, p(f.r_pre), p(f.r_post),
                                      p(a["w_pre"]), p(a["w_post"]), 1, p(a["gate"]), a["scale"], p(dh), p(dn), p(dw_pre),
                                      p(dw_post), p(dgate), p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream))
    for got, ref in ((dh, want.dh), (dn, want.dy), (dw_pre, want.dw_pre), (dw_post, want.dw_post), (dgate, want.dgate)):
        assert torch.equal(got, ref)
    assert ops.status() == M.MOE_OK
