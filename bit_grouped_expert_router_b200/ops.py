"""Operators around the experts, over libmoe (include/moe.h): rows sorted by expert and back
(``dispatch_rows``, ``combine_weighted``), the norms before and after the block (``block_norm``), each with
its gradient, and experts in microscaled 4-bit floating point (``mx4_quantize``, ``mx4_dequantize``,
``mx4_matmul``).

Argument marshalling only, like ``_lib`` (the tensors are checked and passed on by the native module
``_torch_ops``); every step runs in the CUDA library.  The functions take dense, contiguous CUDA tensors of
one device, run there on ``stream`` (default: that device's current stream) without synchronising, and allocate
what they return, and their scratch, on that stream unless an output tensor is given.  A wrong tensor raises
ValueError, a refusal by the library MoeError, memory that runs out torch.OutOfMemoryError; what the kernels find on the
device is kept for ``status``.
Tensors passed with ``stream`` must be ready there and stay alive until the stream has passed the call.  No graph of
automatic differentiation is recorded, not even for tensors that require gradients: the gradients are functions of their
own.  A tensor given to be written counts as modified in place, so a graph that had saved its values refuses to use them.
There is no fallback: if the module has not been built, the first call fails loudly.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib as M
from .build import built_for

_DTYPES = {torch.bfloat16: M.MOE_DTYPE_BF16, torch.float16: M.MOE_DTYPE_FP16, torch.float32: M.MOE_DTYPE_FP32}
_ACTS = {None: M.MOE_ACT_NONE, "swiglu": M.MOE_ACT_SWIGLU}
_x = None   # the native module


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
    """Gradients of the residual, the block's output, the two norms' weights and the gate (None: there was none)."""
    dh: torch.Tensor
    dy: Optional[torch.Tensor]
    dw_pre: Optional[torch.Tensor]
    dw_post: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]


def _ext():
    global _x
    if _x is None:
        M.lib()
        try:
            from . import _torch_ops
        except ImportError as e:
            raise ImportError(f"_torch_ops is not built or does not load ({e}); "
                              "run bit_grouped_expert_router_b200.build.build()") from e
        if _torch_ops.built_for != built_for():
            raise ImportError(f"_torch_ops was built for {_torch_ops.built_for}, this is {built_for()}; "
                              "run bit_grouped_expert_router_b200.build.build()")
        _torch_ops.set_error(M.MoeError)
        _x = _torch_ops
    return _x


def _run(f, stream, *args):
    """f(*args) on `stream`, outputs and scratch allocated there."""
    if stream is None:
        return f(*args)
    for t in args:
        if isinstance(t, torch.Tensor) and t.device != stream.device:
            raise ValueError(f"the stream is of {stream.device}, a tensor of {t.device}")
    with torch.cuda.stream(stream):
        return f(*args)


def _type(dtype) -> int:
    d = _DTYPES.get(dtype)
    if d is None:
        raise ValueError(f"dtype: bf16, fp16 or fp32 is needed, got {dtype}")
    return d


def status(stream=None) -> int:
    """Synchronise the stream (default: the current one) and return the device status code of these operators on its
    device (MOE_OK or MOE_ERR_*); clears it."""
    if stream is None:
        stream = torch.cuda.current_stream()
    with torch.cuda.device(stream.device):
        return int(M.lib().moe_ops_status(stream.cuda_stream))


def dispatch_rows(x, idx, E: int, rows=None, *, stream=None) -> Dispatch:
    """Sort the (token, slot) pairs of idx [T, k] int32 by expert (negative: none) and copy the rows of x [T, H]
    there.  x None: sort only.  Rows behind offsets[E] are left as they are."""
    return Dispatch._make(_run((_x or _ext()).dispatch_rows, stream, x, idx, E, rows))


def dispatch_rows_backward(drows, pos, out=None, *, stream=None):
    """dx [T, H]: for each token the sum of the gradients of its rows."""
    return _run((_x or _ext()).dispatch_rows_backward, stream, drows, pos, out)


def combine_weighted(rows, pos, gates, base=None, out=None, *, stream=None):
    """out [T, H] = base + sum_j gates[:, j] * rows[pos[:, j]] (pos < 0: no row), fp32 sums in slot order."""
    return _run((_x or _ext()).combine_weighted, stream, rows, pos, gates, base, out)


def combine_weighted_backward(dout, rows, pos, gates, drows=None, *, stream=None):
    """(drows, dgates): drows[pos] = gates * dout (other rows as they are), dgates[t, j] = <dout[t], rows[pos[t, j]]>."""
    return _run((_x or _ext()).combine_weighted_backward, stream, dout, rows, pos, gates, drows)


def block_norm(h, y=None, w_pre=None, w_post=None, gate=None, scale: float = 1.0, eps: float = 1e-6,
               norm_post: bool = False, out_dtype=None, h_out=None, n_out=None, pre: bool = True, *,
               stream=None) -> BlockNorm:
    """h' = h + scale * gate * a with a = y (normed if norm_post) * w_post, and n = norm(h') * w_pre (pre False: not
    computed).  y None: the norm of h alone.  out_dtype: n's type without y (default: h's)."""
    n_dtype = -1 if out_dtype is None else _type(out_dtype)
    return BlockNorm._make(_run((_x or _ext()).block_norm, stream, h, y, w_pre, w_post, gate, scale, eps, norm_post,
                                n_dtype, h_out, n_out, pre))


def block_norm_backward(dn, dh_out, h_out, y=None, r_pre=None, r_post=None, w_pre=None, w_post=None, gate=None,
                        scale: float = 1.0, *, stream=None) -> BlockNormGrad:
    """Gradients of block_norm from those of n (dn) and of h' (dh_out), either None, and what the forward call left:
    h_out (h itself where there was no y), y, r_pre and r_post (given: the post norm was taken)."""
    return BlockNormGrad._make(_run((_x or _ext()).block_norm_backward, stream, dn, dh_out, h_out, y, r_pre, r_post,
                                    w_pre, w_post, gate, scale))


def mx4_quantize(x, pos=None, act: Optional[str] = None, codes=None, scales=None, *, stream=None):
    """(codes uint8 [n, K/2], scales uint8 [n, K/32]) of x [T, K] (act "swiglu": of silu(gate) * up for x [T, 2K] =
    [gate | up]); with pos [T, k] each token's row goes to all its places (n = T * k), else row t to row t."""
    if act not in _ACTS:
        raise ValueError(f"act: None or 'swiglu', got {act!r}")
    return _run((_x or _ext()).mx4_quantize, stream, x, pos, _ACTS[act], codes, scales)


def mx4_dequantize(codes, scales, dtype=torch.bfloat16, *, stream=None):
    """The values [..., K] of codes [..., K/2] and scales [..., K/32]."""
    return _run((_x or _ext()).mx4_dequantize, stream, codes, scales, _type(dtype))


def mx4_matmul(codes, scales, w_codes, w_scales, offsets, out=None, dtype=torch.bfloat16, *, stream=None):
    """y [n, N]: each row of the segment offsets[e] .. offsets[e+1] times w_e^T, from rows (codes [n, K/2], scales
    [n, K/32]) and weights (w_codes [E, N, K/2], w_scales [E, N, K/32]) in microscaled 4-bit form.  Rows
    outside the segments are left as they are."""
    return _run((_x or _ext()).mx4_matmul, stream, codes, scales, w_codes, w_scales, offsets, out, _type(dtype))


__all__ = ["Dispatch", "BlockNorm", "BlockNormGrad", "status", "dispatch_rows", "dispatch_rows_backward",
           "combine_weighted", "combine_weighted_backward", "block_norm", "block_norm_backward", "mx4_quantize",
           "mx4_dequantize", "mx4_matmul"]
