"""Operators around the experts, over libmoe (include/moe.h): rows sorted by expert and back
(``dispatch_rows``, ``combine_weighted``), the norms before and after the block (``block_norm``), each with
its gradient, and experts in microscaled 4-bit floating point (``mx4_quantize``, ``mx4_dequantize``,
``mx4_matmul``).

Argument marshalling only, like ``_lib``; every step runs in the CUDA library.  The functions take dense,
contiguous CUDA tensors of one device, run there on ``stream`` (default: that device's current stream)
without synchronising, and allocate what they return, and their scratch, on that stream unless an output tensor is given.
A wrong tensor raises ValueError, a refusal by the library MoeError; what the kernels find on
the device is kept for ``status``.
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional

import torch

from . import _lib as M

_DTYPES = {torch.bfloat16: M.MOE_DTYPE_BF16, torch.float16: M.MOE_DTYPE_FP16, torch.float32: M.MOE_DTYPE_FP32}
_ACTS = {None: M.MOE_ACT_NONE, "swiglu": M.MOE_ACT_SWIGLU}


class Dispatch(NamedTuple):
    """Pairs sorted by expert: rows [T*k, H] (None without x), offsets [E+1], perm [T*k], pos [T, k] int32."""
    rows: Optional[torch.Tensor]
    offsets: torch.Tensor
    perm: torch.Tensor
    pos: torch.Tensor


class BlockNorm(NamedTuple):
    """The new residual h, its norm n, and the row factors (None for what was not computed)."""
    h: Optional[torch.Tensor]
    n: Optional[torch.Tensor]
    r_post: Optional[torch.Tensor]
    r_pre: Optional[torch.Tensor]


class BlockNormGrad(NamedTuple):
    dh: torch.Tensor
    dy: Optional[torch.Tensor]
    dw_pre: Optional[torch.Tensor]
    dw_post: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]


def _placed(f):
    """Runs f with the tensors' device current and, where ``stream`` is given, on that stream."""
    @functools.wraps(f)
    def g(*args, stream=None, **kw):
        t = args[0] if args else None
        if t is None:
            t = next((a for a in (*args, *kw.values()) if isinstance(a, torch.Tensor)), None)
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{f.__name__}: CUDA tensors are needed")
        if stream is not None:
            if stream.device != t.device:
                raise ValueError(f"{f.__name__}: the stream is of {stream.device}, the tensors of {t.device}")
            with torch.cuda.stream(stream):
                return f(*args, **kw)
        if t.get_device() != torch.cuda.current_device():
            with torch.cuda.device(t.device):
                return f(*args, **kw)
        return f(*args, **kw)
    return g


def _stream(t) -> int:
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _have(t, name, dtype, shape, device):
    """t's address, checked (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{device} is needed, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}"
                         f"{'' if t.is_contiguous() else ', not contiguous'}")
    return t.data_ptr()


def _dtype(t, name) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"{name}: bf16, fp16 or fp32 is needed, got {t.dtype}")
    return d


def _matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: a matrix is needed, got shape {tuple(t.shape)}")
    return t.shape


def status(stream=None) -> int:
    """Synchronise the stream (default: the current one) and return the device status code of these operators on its device
    (MOE_OK or MOE_ERR_*); clears it."""
    if stream is None:
        stream = torch.cuda.current_stream()
    with torch.cuda.device(stream.device):
        return int(M.lib().moe_ops_status(stream.cuda_stream))


@_placed
def dispatch_rows(x, idx, E: int, rows=None) -> Dispatch:
    """Sort the (token, slot) pairs of idx [T, k] int32 by expert (negative: none) and copy the rows of x [T, H]
    there.  x None: sort only.  Rows behind offsets[E] are left as they are."""
    T, k = _matrix(idx, "idx")
    dev = idx.get_device()
    ip = _have(idx, "idx", torch.int32, idx.shape, dev)
    H, dt, xp = 8, 0, None
    if x is not None:
        H, dt = _matrix(x, "x")[1], _dtype(x, "x")
        xp = _have(x, "x", x.dtype, (T, H), dev)
        if rows is None:
            rows = x.new_empty((T * k, H))
    elif rows is not None:
        raise ValueError("rows needs x")
    rp = None if rows is None else _have(rows, "rows", x.dtype, (T * k, H), dev)
    offsets = idx.new_empty(max(E, 0) + 1)
    perm = idx.new_empty(T * k)
    pos = idx.new_empty((T, k))
    L = M.lib()
    need = L.moe_dispatch_workspace(T, k, E)
    ws = idx.new_empty(need // 4) if need else None
    M.check(L.moe_dispatch_rows(xp, dt, T, H, ip, k, E, rp, offsets.data_ptr(), perm.data_ptr(), pos.data_ptr(),
                                None if ws is None else ws.data_ptr(), need, _stream(idx)))
    return Dispatch(rows, offsets, perm, pos)


@_placed
def dispatch_rows_backward(drows, pos, out=None):
    """dx [T, H]: for each token the sum of the gradients of its rows."""
    n, H = _matrix(drows, "drows")
    T, k = _matrix(pos, "pos")
    dev = drows.get_device()
    dt = _dtype(drows, "drows")
    dp = _have(drows, "drows", drows.dtype, (n, H), dev)
    pp = _have(pos, "pos", torch.int32, (T, k), dev)
    if out is None:
        out = drows.new_empty((T, H))
    op = _have(out, "out", drows.dtype, (T, H), dev)
    M.check(M.lib().moe_dispatch_rows_backward(dp, dt, n, pp, T, k, H, op, _stream(drows)))
    return out


@_placed
def combine_weighted(rows, pos, gates, base=None, out=None):
    """out [T, H] = base + sum_j gates[:, j] * rows[pos[:, j]] (pos < 0: no row), fp32 sums in slot order."""
    n, H = _matrix(rows, "rows")
    T, k = _matrix(pos, "pos")
    dev = rows.get_device()
    dt = _dtype(rows, "rows")
    rp = _have(rows, "rows", rows.dtype, (n, H), dev)
    pp = _have(pos, "pos", torch.int32, (T, k), dev)
    gp = _have(gates, "gates", torch.float32, (T, k), dev)
    bp = _have(base, "base", rows.dtype, (T, H), dev)
    if out is None:
        out = rows.new_empty((T, H))
    op = _have(out, "out", rows.dtype, (T, H), dev)
    M.check(M.lib().moe_combine_weighted(rp, dt, n, pp, gp, T, k, H, bp, op, _stream(rows)))
    return out


@_placed
def combine_weighted_backward(dout, rows, pos, gates, drows=None):
    """(drows, dgates): drows[pos] = gates * dout (other rows as they are), dgates[t, j] = <dout[t], rows[pos[t, j]]>."""
    n, H = _matrix(rows, "rows")
    T, k = _matrix(pos, "pos")
    dev = rows.get_device()
    dt = _dtype(rows, "rows")
    op = _have(dout, "dout", rows.dtype, (T, H), dev)
    rp = _have(rows, "rows", rows.dtype, (n, H), dev)
    pp = _have(pos, "pos", torch.int32, (T, k), dev)
    gp = _have(gates, "gates", torch.float32, (T, k), dev)
    if drows is None:
        drows = torch.empty_like(rows)
    dp = _have(drows, "drows", rows.dtype, (n, H), dev)
    dgates = gates.new_empty((T, k))
    M.check(M.lib().moe_combine_weighted_backward(op, dt, rp, n, pp, gp, T, k, H, dp, dgates.data_ptr(), _stream(rows)))
    return drows, dgates


@_placed
def block_norm(h, y=None, w_pre=None, w_post=None, gate=None, scale: float = 1.0, eps: float = 1e-6,
               norm_post: bool = False, out_dtype=None, h_out=None, n_out=None, pre: bool = True) -> BlockNorm:
    """h' = h + scale * gate * a with a = y (normed if norm_post) * w_post, and n = norm(h') * w_pre (pre False: not
    computed).  y None: the norm of h alone.  out_dtype: n's type without y (default: h's)."""
    T, H = _matrix(h, "h")
    dev = h.get_device()
    hd = _dtype(h, "h")
    hp = _have(h, "h", h.dtype, (T, H), dev)
    nt = y.dtype if y is not None else h.dtype if out_dtype is None else out_dtype
    yd = _DTYPES.get(nt)
    if yd is None:
        raise ValueError(f"y: bf16, fp16 or fp32 is needed, got {nt}")
    if out_dtype is not None and out_dtype is not nt:
        raise ValueError(f"n has y's type ({nt}), not {out_dtype}")
    yp = _have(y, "y", nt, (T, H), dev)
    wp, wq = _have(w_pre, "w_pre", torch.float32, (H,), dev), _have(w_post, "w_post", torch.float32, (H,), dev)
    gp = _have(gate, "gate", torch.float32, (T,), dev)
    if y is not None and h_out is None:
        h_out = torch.empty_like(h)
    if pre and n_out is None:
        n_out = h.new_empty((T, H), dtype=nt)
    op, np_ = _have(h_out, "h_out", h.dtype, (T, H), dev), _have(n_out, "n_out", nt, (T, H), dev)
    r_post = h.new_empty(T, dtype=torch.float32) if norm_post else None
    r_pre = h.new_empty(T, dtype=torch.float32) if pre else None
    M.check(M.lib().moe_block_norm(hp, hd, yp, yd, T, H, wq, 1 if norm_post else 0, gp, scale, wp, eps, op, np_,
                                   None if r_post is None else r_post.data_ptr(),
                                   None if r_pre is None else r_pre.data_ptr(), _stream(h)))
    return BlockNorm(h_out, n_out, r_post, r_pre)


@_placed
def block_norm_backward(dn, dh_out, h_out, y=None, r_pre=None, r_post=None, w_pre=None, w_post=None, gate=None,
                        scale: float = 1.0) -> BlockNormGrad:
    """Gradients of block_norm from those of n (dn) and of h' (dh_out), either None, and what the forward call left:
    h_out (h itself where there was no y), y, r_pre and r_post (given: the post norm was taken)."""
    if h_out is None:
        raise ValueError("h_out is needed")
    T, H = _matrix(h_out, "h_out")
    dev = h_out.get_device()
    hd, nt = _dtype(h_out, "h_out"), (y if y is not None else dn if dn is not None else h_out).dtype
    yd = _DTYPES.get(nt)
    if yd is None:
        raise ValueError(f"y: bf16, fp16 or fp32 is needed, got {nt}")
    np_, ip = _have(dn, "dn", nt, (T, H), dev), _have(dh_out, "dh_out", h_out.dtype, (T, H), dev)
    hp, yp = _have(h_out, "h_out", h_out.dtype, (T, H), dev), _have(y, "y", nt, (T, H), dev)
    rp, rq = _have(r_pre, "r_pre", torch.float32, (T,), dev), _have(r_post, "r_post", torch.float32, (T,), dev)
    wp, wq = _have(w_pre, "w_pre", torch.float32, (H,), dev), _have(w_post, "w_post", torch.float32, (H,), dev)
    gp = _have(gate, "gate", torch.float32, (T,), dev)
    dh = torch.empty_like(h_out)
    dy = torch.empty_like(y) if y is not None else None
    dw_pre = w_pre.new_empty(H) if w_pre is not None else None
    dw_post = w_post.new_empty(H) if w_post is not None else None
    dgate = gate.new_empty(T) if gate is not None else None
    L = M.lib()
    need = L.moe_block_norm_backward_workspace(T, H) if dw_pre is not None or dw_post is not None else 0
    ws = h_out.new_empty(need // 4, dtype=torch.float32) if need else None
    M.check(L.moe_block_norm_backward(np_, ip, hp, hd, yp, yd, T, H, rp, rq, wp, wq, 0 if r_post is None else 1, gp, scale,
                                      dh.data_ptr(), M._ptr(dy), M._ptr(dw_pre), M._ptr(dw_post), M._ptr(dgate),
                                      M._ptr(ws), need, _stream(h_out)))
    return BlockNormGrad(dh, dy, dw_pre, dw_post, dgate)


@_placed
def mx4_quantize(x, pos=None, act: Optional[str] = None, codes=None, scales=None):
    """(codes uint8 [n, K/2], scales uint8 [n, K/32]) of x [T, K] (act "swiglu": of silu(gate) * up for x [T, 2K] =
    [gate | up]); with pos [T, k] each token's row goes to all its places (n = T * k), else row t to row t."""
    T, W = _matrix(x, "x")
    if act not in _ACTS:
        raise ValueError(f"act: None or 'swiglu', got {act!r}")
    K = W // 2 if act == "swiglu" else W
    if act == "swiglu" and W % 2:
        raise ValueError("swiglu needs rows of an even width")
    dev = x.get_device()
    xp = _have(x, "x", x.dtype, (T, W), dev)
    k = 1 if pos is None else _matrix(pos, "pos")[1]
    pp = _have(pos, "pos", torch.int32, (T, k), dev)
    n = T * k if codes is None else _matrix(codes, "codes")[0]
    if codes is None:
        codes = x.new_empty((n, K // 2), dtype=torch.uint8)
    if scales is None:
        scales = x.new_empty((n, K // 32), dtype=torch.uint8)
    cp = _have(codes, "codes", torch.uint8, (n, K // 2), dev)
    sp = _have(scales, "scales", torch.uint8, (n, K // 32), dev)
    M.check(M.lib().moe_mx4_quantize(xp, _dtype(x, "x"), T, K, _ACTS[act], pp, k, n, cp, sp, _stream(x)))
    return codes, scales


@_placed
def mx4_dequantize(codes, scales, dtype=torch.bfloat16):
    """The values [..., K] of codes [..., K/2] and scales [..., K/32]."""
    dev = codes.get_device()
    K = 2 * codes.shape[-1]
    cp = _have(codes, "codes", torch.uint8, codes.shape, dev)
    sp = _have(scales, "scales", torch.uint8, codes.shape[:-1] + (K // 32,), dev)
    if dtype not in _DTYPES:
        raise ValueError(f"dtype: bf16, fp16 or fp32 is needed, got {dtype}")
    out = codes.new_empty(codes.shape[:-1] + (K,), dtype=dtype)
    M.check(M.lib().moe_mx4_dequantize(cp, sp, out.numel() // K if K else 0, K, out.data_ptr(), _DTYPES[dtype],
                                       _stream(codes)))
    return out


@_placed
def mx4_matmul(codes, scales, w_codes, w_scales, offsets, out=None, dtype=torch.bfloat16):
    """y [n, N]: each row of the segment offsets[e] .. offsets[e+1] times w_e^T, from rows (codes [n, K/2], scales
    [n, K/32]) and weights (w_codes [E, N, K/2], w_scales [E, N, K/32]) in microscaled 4-bit form.  Rows
    outside the segments are left as they are."""
    n, Kh = _matrix(codes, "codes")
    if w_codes.dim() != 3:
        raise ValueError(f"w_codes: [E, N, K/2] is needed, got shape {tuple(w_codes.shape)}")
    E, N = w_codes.shape[:2]
    dev = codes.get_device()
    cp = _have(codes, "codes", torch.uint8, (n, Kh), dev)
    sp = _have(scales, "scales", torch.uint8, (n, Kh // 16), dev)
    wp = _have(w_codes, "w_codes", torch.uint8, (E, N, Kh), dev)
    wq = _have(w_scales, "w_scales", torch.uint8, (E, N, Kh // 16), dev)
    fp = _have(offsets, "offsets", torch.int32, (E + 1,), dev)
    if out is None:
        if dtype not in _DTYPES:
            raise ValueError(f"dtype: bf16 or fp32 is needed, got {dtype}")
        out = codes.new_empty((n, N), dtype=dtype)
    op = _have(out, "out", out.dtype, (n, N), dev)
    M.check(M.lib().moe_mx4_matmul(cp, sp, n, 2 * Kh, wp, wq, E, N, fp, op, _dtype(out, "out"), _stream(codes)))
    return out


__all__ = ["Dispatch", "BlockNorm", "BlockNormGrad", "status", "dispatch_rows", "dispatch_rows_backward",
           "combine_weighted", "combine_weighted_backward", "block_norm", "block_norm_backward", "mx4_quantize",
           "mx4_dequantize", "mx4_matmul"]
