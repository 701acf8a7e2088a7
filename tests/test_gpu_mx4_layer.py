"""Experts in microscaled 4-bit floating point as a layer: Mx4Experts and the expert-parallel Mx4Shard against the same
steps in 64 bits, a block of norms, router, experts and residual, and a training step through the operators."""
import threading

import numpy as np
import pytest
import torch

import ops_plain as P
from bit_grouped_expert_router_b200 import _lib as M
from bit_grouped_expert_router_b200 import build as B
from bit_grouped_expert_router_b200 import ops, synth
from bit_grouped_expert_router_b200.ep import Exchange, ExpertParallelLayer, Mx4Shard
from bit_grouped_expert_router_b200.mx4 import Mx4Experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.build()
    M.lib()


def make(E, H, I, seed):
    g = torch.Generator().manual_seed(seed)
    w = [torch.randn(s, generator=g) * s[2] ** -0.5 for s in ((E, I, H), (E, I, H), (E, H, I))]
    return Mx4Experts.from_dense(*[t.cuda() for t in w])


def values(packed):
    return P.mx4_values(packed[0].cpu(), packed[1].cpu())


def plain(ex, x, idx, gates, base=None):
    """The layer's steps in 64 bits, rounded to bf16 where the layer stores bf16."""
    wgu, wd = values(ex.gateup), values(ex.down)
    c, s = P.mx4_quantize(x.double())
    xq = P.mx4_values(P.mx4_pack(c), s)
    out = torch.zeros((x.shape[0], ex.H), dtype=torch.float64) if base is None else base.double()
    for t in range(x.shape[0]):
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            if e < 0:
                continue
            h = (wgu[e] @ xq[t]).to(torch.bfloat16).double()
            a = h[:ex.I] * torch.sigmoid(h[:ex.I]) * h[ex.I:]
            c, s = P.mx4_quantize(a.view(1, -1))
            y = wd[e] @ P.mx4_values(P.mx4_pack(c), s)[0]
            out[t] += float(gates[t, j]) * y.to(torch.bfloat16).double()
    return out


def close(got, want):
    """Equal but for the roundings of the sums: fp32 sums put about one bf16 value in a thousand on its other side
    (2^-16 against 2^-8 of a step), one such value in thirty then crosses a border of the 4-bit grid (a quarter of it): a
    relative error of sqrt(3e-5) / 4, 1.4e-3, next to 2^-9 from the result's own rounding.  1e-2 leaves room for neither a
    wrong scale (a factor of two in 32 values) nor a wrong row."""
    g = got.cpu().double()
    assert torch.isfinite(g).all()
    assert float((g - want).norm() / want.norm()) < 1e-2


@pytest.mark.parametrize("E,H,I,T,k", [(4, 64, 32, 1, 2), (8, 256, 128, 37, 3), (5, 320, 96, 130, 4), (256, 512, 64, 3, 8)])
def test_experts_match_the_plain_steps(E, H, I, T, k):
    ex = make(E, H, I, E + T)
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16)
    idx = torch.rand((T, E), generator=g).topk(k, dim=1)[1].to(torch.int32)
    if T > 10:
        idx[3, 1] = -1
        idx[7] = -1
    gates = torch.rand((T, k), generator=g)
    base = torch.randn((T, H), generator=g).to(torch.bfloat16)
    close(ex.forward(x.cuda(), idx.cuda(), gates.cuda()), plain(ex, x, idx, gates))
    got = ex.forward(x.cuda(), idx.cuda(), gates.cuda(), base=base.cuda())
    close(got, plain(ex, x, idx, gates, base))
    if T > 10:
        assert torch.equal(got[7].cpu(), base[7])          # a token without an expert keeps its base
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = ex.forward(x.cuda(), idx.cuda(), gates.cuda(), base=base.cuda(), stream=s)
    torch.cuda.synchronize()
    assert torch.equal(again, got)
    assert ex.forward(x[:0].cuda(), idx[:0].cuda(), gates[:0].cuda()).shape == (0, H)
    assert ops.status() == M.MOE_OK


def test_experts_of_other_sizes_are_refused():
    a, b = make(2, 64, 32, 1), make(2, 96, 32, 2)
    with pytest.raises(ValueError):
        Mx4Experts(a.gateup, b.down)


def test_block_of_norm_router_experts_and_residual():
    """One block as a model runs it: norm, router (libmoe handle), experts, weighted sum, residual and the next norm."""
    shape = synth.Shape("block", T=60, H=256, E=16, k=4, I=128, has_shared=False, seed=61)
    w = synth.make_layer(shape)
    router = M.Layer.from_shape({n: v.cuda() if v is not None else None for n, v in w.items()}, shape, max_tokens=64,
                                flags=M.MOE_FLAG_NO_EXPERTS)
    ex = make(shape.E, shape.H, shape.I, 3)
    g = torch.Generator().manual_seed(6)
    h = torch.randn((shape.T, shape.H), generator=g).to(torch.bfloat16)
    w1, w2 = 1 + 0.1 * torch.randn(shape.H, generator=g), 1 + 0.1 * torch.randn(shape.H, generator=g)
    first = ops.block_norm(h.cuda(), w_pre=w1.cuda())
    r = router.route(first.n)
    y = ex.forward(first.n, r["idx"], r["gates"])
    last = ops.block_norm(h.cuda(), y, w_pre=w2.cuda(), scale=0.5)
    torch.cuda.synchronize()
    assert router.status() == M.MOE_OK and ops.status() == M.MOE_OK
    want = P.block_norm(h, None, w1, None, None, 1.0, 1e-6, False)
    P.rounded(first.n, *want["n"], "n")
    ref = plain(ex, first.n.cpu(), r["idx"].cpu(), r["gates"].cpu())
    close(y, ref)
    want = P.block_norm(h, y.cpu(), w2, None, None, 0.5, 1e-6, False)
    P.rounded(last.h, *want["h"], "h")
    P.rounded(last.n, *want["n"], "n")
    router.close()


class ThreadExchange(Exchange):
    """All-to-all between shards run as threads of one process: host-side hand-offs between two barriers."""

    def __init__(self, rank, world, board, barrier):
        super().__init__(None, world)
        self.rank, self.board, self.barrier = rank, board, barrier

    def _swap(self, parts):
        self.board[self.rank] = parts
        self.barrier.wait()
        got = [self.board[r][self.rank] for r in range(self.world)]
        self.barrier.wait()
        return got

    def counts(self, send_counts):
        return torch.stack(self._swap(list(send_counts.unbind(0))))

    def rows(self, send, send_splits, recv_splits, out=None):
        return torch.cat(self._swap(list(torch.split(send, list(send_splits)))), 0)


def test_expert_parallel_shards_equal_one_rank():
    shape = synth.Shape("mx4ep", T=90, H=256, E=16, k=3, I=64, seed=62)
    w = {n: v.cuda() if v is not None else None for n, v in synth.make_layer(shape).items()}
    full, shared = make(16, 256, 64, 9), make(1, 256, 64, 10)
    x_host = synth.make_x(shape)
    x = x_host.cuda()

    def run(world):
        cuts = [shape.T * r // world for r in range(world + 1)]
        board, barrier, outs, errs = {}, threading.Barrier(world), [None] * world, []
        n = 16 // world
        part = lambda p, r: tuple(t[r * n:(r + 1) * n].contiguous() for t in p)  # noqa: E731
        shards = [Mx4Shard(w, Mx4Experts(part(full.gateup, r), part(full.down, r)), shared, 16, 3, world) for r in range(world)]

        def one(r):
            try:
                outs[r] = ExpertParallelLayer(shards[r], ThreadExchange(r, world, board, barrier)).forward(
                    x_host[cuts[r]:cuts[r + 1]].cuda())
                torch.cuda.synchronize()
            except BaseException as e:
                errs.append(e)
                barrier.abort()

        threads = [threading.Thread(target=one, args=(r,)) for r in range(world)]
        [t.start() for t in threads]
        [t.join(timeout=300) for t in threads]
        for s in shards:
            s.close()
        if errs:
            raise errs[0]
        return torch.cat(outs)

    one = run(1)
    assert torch.equal(run(2), one)
    router = M.Layer.from_shape(w, shape, max_tokens=128, flags=M.MOE_FLAG_NO_EXPERTS)
    r = router.route(x)
    base = shared.forward(x, torch.zeros((shape.T, 1), dtype=torch.int32, device="cuda"), r["shared_gate"].view(-1, 1))
    y = full.forward(x, r["idx"], r["gates"], base=base)
    # each rank rounds a row's weighted result to bf16 before the sum over k, one rank's forward only after it
    g, ref = one.double().cpu().numpy(), y.double().cpu().numpy()
    assert np.linalg.norm(g - ref) / np.linalg.norm(ref) < 2 * 2.0 ** -8
    router.close()
    assert ops.status() == M.MOE_OK


def test_training_step_through_the_operators():
    """Norm, dispatch, dense experts, weighted sum, residual: gradients of every input against automatic differentiation
    in 64 bits.  All steps run in fp32; a step's error is at most some 100 roundings (2^-24) of its magnitudes, and the
    deepest gradient passes five steps, so 1e-4 of each gradient's largest value covers them."""
    g = torch.Generator().manual_seed(12)
    T, k, E, H = 50, 3, 6, 64
    idx = torch.rand((T, E), generator=g).topk(k, dim=1)[1].to(torch.int32)
    idx[4, 0] = -1
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    h, gates, w1, w2, we = rand(T, H), torch.rand((T, k), generator=g), 1 + 0.1 * rand(H), 1 + 0.1 * rand(H), rand(E, H, H) / 8
    tgate, loss_n, loss_h = torch.rand(T, generator=g), rand(T, H), rand(T, H)
    c = lambda t: t.cuda()  # noqa: E731

    first = ops.block_norm(c(h), w_pre=c(w1))
    d = ops.dispatch_rows(first.n, c(idx), E)
    ends = d.offsets.tolist()
    y = torch.zeros_like(d.rows)
    for e in range(E):
        y[ends[e]:ends[e + 1]] = d.rows[ends[e]:ends[e + 1]] @ c(we[e])
    m = ops.combine_weighted(y, d.pos, c(gates))
    last = ops.block_norm(c(h), m, w_pre=c(w2), w_post=c(w1), gate=c(tgate), scale=0.3, norm_post=True)
    b2 = ops.block_norm_backward(c(loss_n), c(loss_h), last.h, m, r_pre=last.r_pre, r_post=last.r_post, w_pre=c(w2),
                                 w_post=c(w1), gate=c(tgate), scale=0.3)
    dy, dgates = ops.combine_weighted_backward(b2.dy, y, d.pos, c(gates))
    drows = torch.zeros_like(dy)
    for e in range(E):
        drows[ends[e]:ends[e + 1]] = dy[ends[e]:ends[e + 1]] @ c(we[e]).t()
    dn = ops.dispatch_rows_backward(drows, d.pos)
    b1 = ops.block_norm_backward(dn, b2.dh, c(h), r_pre=first.r_pre, w_pre=c(w1))

    v = {n: t.double().requires_grad_() for n, t in dict(h=h, gates=gates, w1=w1, w2=w2, tgate=tgate).items()}
    norm = lambda t: t / torch.sqrt((t * t).mean(1, keepdim=True) + float(torch.tensor(1e-6)))  # noqa: E731
    n1 = norm(v["h"]) * v["w1"]
    mm = torch.zeros((T, H), dtype=torch.float64)
    for j in range(k):
        e = idx[:, j].long()
        mm = mm + torch.where(e.view(-1, 1) >= 0, v["gates"][:, j:j + 1] * torch.einsum("th,thn->tn", n1, we.double()[e.clamp(min=0)]), 0.0)
    h2 = v["h"] + float(torch.tensor(0.3)) * v["tgate"].view(-1, 1) * norm(mm) * v["w1"]
    ((norm(h2) * v["w2"] * loss_n.double()).sum() + (h2 * loss_h.double()).sum()).backward()
    for name, got in (("h", b1.dh), ("gates", dgates), ("w2", b2.dw_pre), ("w1", b2.dw_post + b1.dw_pre), ("tgate", b2.dgate)):
        ref = v[name].grad
        assert float((got.cpu().double() - ref).abs().max()) <= 1e-4 * float(ref.abs().max()), name
