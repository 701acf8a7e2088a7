"""Host-side checks of the operators around the experts (no GPU needed): each entry point refuses bad
arguments before it touches the device, and the Python calls refuse tensors they cannot pass on."""
import ctypes
import inspect
import os
import sys
import sysconfig

import pytest
import torch

import ops_plain as P
from bit_grouped_expert_router_b200 import _lib as M
from bit_grouped_expert_router_b200 import build as B
from bit_grouped_expert_router_b200 import ops

A = 0x1000   # an aligned address; never dereferenced: the argument checks and the device check come first
BF16, FP16, FP32 = M.MOE_DTYPE_BF16, M.MOE_DTYPE_FP16, M.MOE_DTYPE_FP32
CALLS = {
    "moe_dispatch_rows": dict(x=A, dtype=BF16, T=4, H=64, idx=A, k=2, E=8, rows=A, offsets=A, perm=A, pos=A, ws=None,
                              ws_bytes=0, stream=None),
    "moe_dispatch_rows_backward": dict(drows=A, dtype=BF16, n_rows=8, pos=A, T=4, k=2, H=64, dx=A, stream=None),
    "moe_combine_weighted": dict(rows=A, dtype=BF16, n_rows=8, pos=A, gates=A, T=4, k=2, H=64, base=None, out=A,
                                 stream=None),
    "moe_combine_weighted_backward": dict(dout=A, dtype=BF16, rows=A, n_rows=8, pos=A, gates=A, T=4, k=2, H=64,
                                          drows=A, dgates=A, stream=None),
    "moe_block_norm": dict(h=A, h_dtype=BF16, y=A, y_dtype=BF16, T=4, H=64, w_post=A, norm_post=1, gate=A, scale=1.0,
                           w_pre=A, eps=1e-6, h_out=A, n_out=A, r_post=A, r_pre=A, stream=None),
    "moe_block_norm_backward": dict(dn=A, dh_out=A, h_out=A, h_dtype=BF16, y=A, y_dtype=BF16, T=4, H=64, r_pre=A,
                                    r_post=A, w_pre=A, w_post=A, norm_post=1, gate=A, scale=1.0, dh=A, dy=A, dw_pre=A,
                                    dw_post=A, dgate=A, ws=A, ws_bytes=1 << 20, stream=None),
    "moe_mx4_quantize": dict(x=A, dtype=BF16, T=4, K=64, act=0, pos=None, k=1, n_rows=4, codes=A, scales=A, stream=None),
    "moe_mx4_dequantize": dict(codes=A, scales=A, rows=4, K=64, out=A, dtype=BF16, stream=None),
    "moe_mx4_matmul": dict(codes=A, scales=A, n_rows=4, K=64, w_codes=A, w_scales=A, E=2, N=16, offsets=A, y=A,
                           dtype=BF16, stream=None),
}
BAD = {
    "moe_dispatch_rows": [dict(dtype=3), dict(T=-1), dict(H=0), dict(H=12), dict(H=65544), dict(k=0), dict(k=33), dict(E=0),
                          dict(E=257), dict(x=None), dict(rows=None), dict(x=A + 8), dict(idx=None), dict(idx=A + 2),
                          dict(offsets=None), dict(perm=None), dict(pos=None), dict(T=1 << 29, k=2),
                          dict(T=4096, ws=None), dict(T=4096, ws=A, ws_bytes=16), dict(T=4096, ws=A + 4, ws_bytes=1 << 30)],
    "moe_dispatch_rows_backward": [dict(dtype=-1), dict(T=-1), dict(H=4), dict(k=0), dict(n_rows=-1), dict(drows=None),
                                   dict(pos=None), dict(dx=None), dict(dx=A + 4)],
    "moe_combine_weighted": [dict(dtype=9), dict(H=20), dict(k=40), dict(gates=None), dict(gates=A + 1), dict(rows=None),
                             dict(base=A + 8), dict(out=None), dict(n_rows=-3)],
    "moe_combine_weighted_backward": [dict(dtype=9), dict(H=20), dict(gates=None), dict(rows=None), dict(dout=None),
                                      dict(drows=None), dict(dgates=None), dict(drows=A + 2)],
    "moe_block_norm": [dict(h_dtype=5), dict(y_dtype=5), dict(h_dtype=FP16), dict(h_dtype=BF16, y_dtype=FP32), dict(T=-1),
                       dict(H=7), dict(H=16392), dict(norm_post=2), dict(eps=-1.0), dict(eps=float("nan")), dict(h=None),
                       dict(y=None), dict(h=A + 8), dict(w_post=A + 4), dict(norm_post=0), dict(n_out=A + 2)],
    "moe_block_norm_backward": [dict(h_dtype=FP16), dict(H=12), dict(dn=None), dict(h_out=None), dict(r_pre=None),
                                dict(r_post=None), dict(y=None), dict(ws=None), dict(ws_bytes=64), dict(dy=A + 8),
                                dict(dw_pre=A + 4), dict(norm_post=-1)],
    "moe_mx4_quantize": [dict(dtype=4), dict(T=-1), dict(K=16), dict(K=48), dict(K=65568), dict(act=2), dict(n_rows=3),
                         dict(pos=A, k=0), dict(pos=A, k=33), dict(x=None), dict(codes=None), dict(scales=A + 1),
                         dict(pos=A + 1)],
    "moe_mx4_dequantize": [dict(dtype=4), dict(rows=-1), dict(K=40), dict(codes=None), dict(out=A + 2)],
    "moe_mx4_matmul": [dict(dtype=FP16), dict(n_rows=-1), dict(K=33), dict(E=0), dict(E=257), dict(N=12), dict(N=0),
                       dict(E=256, N=1 << 23), dict(codes=None), dict(w_codes=A + 8), dict(offsets=None), dict(y=None)],
}


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.lib()


@pytest.mark.parametrize("name,change", [(n, c) for n in BAD for c in BAD[n]], ids=str)
def test_bad_arguments_are_refused_before_the_device(lib, name, change):
    rc = getattr(lib, name)(*{**CALLS[name], **change}.values())
    assert rc == M.MOE_ERR_INVALID_ARG
    assert lib.moe_last_error().decode()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
@pytest.mark.parametrize("name", CALLS)
def test_good_arguments_reach_the_device_check(lib, name):
    assert getattr(lib, name)(*CALLS[name].values()) == M.MOE_ERR_CUDA
    assert lib.moe_ops_status(None) == M.MOE_ERR_CUDA


@pytest.mark.parametrize("name", [n for n in CALLS if n not in ("moe_dispatch_rows", "moe_block_norm_backward")])
def test_no_rows_is_a_no_op(lib, name):
    """Empty tensors have no address: nothing but sizes is looked at, and nothing launched."""
    call = {n: None if v == A else v for n, v in CALLS[name].items()}
    for n in ("T", "n_rows", "rows"):
        if n in call and (n != "rows" or name == "moe_mx4_dequantize"):
            call[n] = 0
    assert getattr(lib, name)(*call.values()) == M.MOE_OK, lib.moe_last_error()


def test_workspace_sizes(lib):
    assert lib.moe_dispatch_workspace(512, 8, 256) == 0             # 4096 pairs: sorted without scratch
    assert lib.moe_dispatch_workspace(513, 8, 256) == 5 * 256 * 4   # a count per chunk of 1024 pairs and expert
    n = lib.moe_dispatch_workspace(1 << 24, 32, 256)                # 2^29 pairs: the chunks grow, not their number
    assert 0 < n <= 256 * 256 * 4
    assert lib.moe_dispatch_workspace(-1, 8, 256) == lib.moe_dispatch_workspace(8, 8, 300) == 0
    assert lib.moe_block_norm_backward_workspace(1, 2048) == 2 * 2048 * 4
    assert lib.moe_block_norm_backward_workspace(4, 12) == 0


def test_python_calls_refuse_what_they_cannot_pass_on(lib):
    cpu, idx = torch.zeros((2, 64)), torch.zeros((2, 2), dtype=torch.int32)
    for call in (lambda: ops.dispatch_rows(cpu, idx, 4), lambda: ops.dispatch_rows_backward(cpu, idx),
                 lambda: ops.combine_weighted(cpu, idx, cpu), lambda: ops.combine_weighted_backward(cpu, cpu, idx, cpu),
                 lambda: ops.block_norm(cpu), lambda: ops.block_norm_backward(cpu, None, cpu), lambda: ops.mx4_quantize(cpu),
                 lambda: ops.mx4_dequantize(cpu, cpu), lambda: ops.mx4_matmul(cpu, cpu, cpu, cpu, idx)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="idx: a tensor"):
        ops.dispatch_rows(cpu, None, 4)
    with pytest.raises(ValueError, match="h_out: a tensor"):
        ops.block_norm_backward(cpu, None, None)
    with pytest.raises(ValueError, match="act: an integer"):
        ops._ext().mx4_quantize(cpu, None, "four", None, None)
    with pytest.raises(ValueError, match="act"):
        ops.mx4_quantize(cpu, act="gelu")
    for dtype in (torch.float64, torch.uint8):
        with pytest.raises(ValueError, match="dtype"):
            ops.mx4_dequantize(cpu, cpu, dtype=dtype)
    with pytest.raises(ValueError, match="arguments"):
        ops._ext().combine_weighted(cpu)


def test_the_native_module_shares_the_loaded_libstdcxx(lib):
    with open(B.EXT, "rb") as f:
        assert b"libstdc++.so.6" in f.read()      # a needed library, not a copy inside


def test_every_operator_takes_a_stream_and_is_documented():
    for n in ops.__all__:
        f = getattr(ops, n)
        assert f.__doc__, n
        if inspect.isfunction(f):
            assert "stream" in inspect.signature(f).parameters, n


# ---- the plain forms themselves --------------------------------------------------------------------
def test_plain_quantisation_is_the_nearest_value():
    g = torch.Generator().manual_seed(3)
    v = torch.randn((40, 64), generator=g, dtype=torch.float64)
    c, s = P.mx4_quantize(v)
    got = P.mx4_values(P.mx4_pack(c), s.to(torch.uint8))
    unit = torch.exp2(s.double() - 127).repeat_interleave(32, dim=1)
    all_values = torch.tensor(P.MAGNITUDES + [-m for m in P.MAGNITUDES], dtype=torch.float64)
    nearest = (v.unsqueeze(-1) - all_values * unit.unsqueeze(-1)).abs().amin(-1)
    assert torch.equal((v - got).abs(), nearest)
    top = (v.abs() / unit).view(40, 2, 32).amax(-1)
    assert ((top >= 4) & (top < 8)).all()


def test_plain_norm_gradient_is_the_difference_quotient():
    g = torch.Generator().manual_seed(5)
    T, H = 3, 16
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    a = dict(h=r(T, H), y=r(T, H), w_pre=r(H), w_post=r(H), gate=r(T), scale=0.5, eps=1e-6, norm_post=True)
    dn, dh = r(T, H), r(T, H)
    o = P.block_norm(**a)
    grad = P.block_norm_backward(dn, dh, o["h"][0], a["y"], o["r_pre"][0], o["r_post"][0], a["w_pre"], a["w_post"],
                                 a["gate"], a["scale"])
    loss = lambda **c: float((P.block_norm(**{**a, **c})["n"][0] * dn + P.block_norm(**{**a, **c})["h"][0] * dh).sum())  # noqa: E731
    for name, of in (("h", "dh"), ("y", "dy"), ("gate", "dgate"), ("w_post", "dw_post"), ("w_pre", "dw_pre")):
        for at in range(a[name].numel()):
            up, down = a[name].clone(), a[name].clone()
            up.view(-1)[at] += 1e-5
            down.view(-1)[at] -= 1e-5
            # central differences: 1e-10 of a third derivative, and 1e-16 / 1e-5 of the loss
            assert abs((loss(**{name: up}) - loss(**{name: down})) / 2e-5 - float(grad[of][0].reshape(-1)[at])) < 1e-6


def test_experts_refuse_a_stream_of_another_device(lib):
    """As each operator does: the steps would run on the tensors' device, on a stream that nobody waits for."""
    from types import SimpleNamespace

    from bit_grouped_expert_router_b200.mx4 import Mx4Experts
    packed = lambda n, k: (torch.zeros((2, n, k // 2), dtype=torch.uint8), torch.zeros((2, n, k // 32), dtype=torch.uint8))  # noqa: E731
    ex = Mx4Experts(packed(64, 64), packed(64, 32))
    x, idx, gates = torch.zeros((3, 64)), torch.zeros((3, 1), dtype=torch.int32), torch.zeros((3, 1))
    other = SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="the stream is of cuda:1, a tensor of cpu"):
        ex.forward(x, idx, gates, stream=other)


@pytest.fixture
def small_tree(tmp_path, monkeypatch):
    """The build pointed at a tree of one small source."""
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "one.cu").write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    (src / "torch_ops.cpp").write_text("#error this module does not compile\n")
    for name, value in dict(CSRC=str(src), BUILD=str(tmp_path / "obj"), LIB=str(tmp_path / "libmoe.so"), SOURCES=["one.cu"],
                            PKG=str(tmp_path), EXT=str(tmp_path / os.path.basename(B.EXT))).items():
        monkeypatch.setattr(B, name, value)
    return tmp_path


def test_the_library_is_built_where_its_torch_module_does_not_compile(small_tree):
    """The C ABI needs nvcc only; the module's failure is told all the same, and again on the next call, and a module of an
    older source does not stay behind."""
    for _ in range(2):
        with open(B.EXT, "w"):
            os.utime(B.EXT, (0, 0))
        with pytest.warns(RuntimeWarning, match="torch_ops.cpp failed"):
            assert B.build() == B.LIB
        assert ctypes.CDLL(B.LIB).one() == 1
        assert not B.up_to_date() and not os.path.exists(B.EXT)


def test_the_library_is_built_without_torch(small_tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)      # import torch raises ImportError
    assert B.build() == B.LIB
    assert ctypes.CDLL(B.LIB).one() == 1
    made = os.stat(B.LIB).st_mtime_ns
    B.build()
    assert os.stat(B.LIB).st_mtime_ns == made            # nothing left to build


def test_a_module_of_another_torch_or_python_is_not_taken(lib, monkeypatch):
    """Its classes and calls are those of the torch and the Python it was compiled against."""
    assert B.EXT.endswith(sysconfig.get_config_var("EXT_SUFFIX"))      # another Python does not find it
    assert B.up_to_date()
    monkeypatch.setattr(ops, "_x", None)
    assert ops._ext().built_for == f"torch {torch.__version__}"
    monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    assert not B.up_to_date()
    monkeypatch.setattr(ops, "_x", None)
    with pytest.raises(ImportError, match="1.0.0.other"):
        ops._ext()
