"""The operators around the routed layer (include/moe.h, same names): the norms and residual of the decoder
block, int8 products for its shared expert, bf16 experts grouped by the routing.

Argument marshalling only, most of it compiled (csrc/python_ops.cpp, built as _ops next to libmoe.so).  All
tensors of a call are on one CUDA device, which need not be the current one; the work is enqueued on that
device's current stream, or on `stream`, in which case outputs are allocated for that stream and inputs are
recorded on it.  Two new outputs of a call that take up to 1 MB together share one allocation (each is contiguous
and starts on a multiple of 512 bytes).  Tensors of another type, shape, layout or device raise ValueError (TypeError if
they are no tensors), what the C ABI refuses raises MoEError.  Inference only, like the layer: outputs have no autograd
history, whatever the inputs require."""
from __future__ import annotations

import torch

from ._lib import MoEError, load

load()


class _Unbuilt:
    """In the place of _ops where it is missing or does not load: the layer needs only libmoe.so, and so does importing the
    package; the functions below raise."""

    def __init__(self, cause):
        self._cause = cause

    def __getattr__(self, name):
        raise ImportError("_ops.so not built, or not for this torch: run `python decode_moe_layer_b200/build.py`") \
            from self._cause


try:
    from . import _ops  # (resolves its symbols in libmoe.so)
    _ops.raise_as(MoEError)
except ImportError as e:
    _ops = _Unbuilt(e)


def _on(stream, fn, *args):
    """fn on `stream`: its outputs come from that stream's pool, its tensors are recorded on it."""
    dev = args[0].device if isinstance(args[0], torch.Tensor) else None
    if dev is not None and stream.device != dev:
        raise ValueError("stream is on %s, the tensors are on %s" % (stream.device, dev))
    with torch.cuda.stream(stream):
        res = fn(*args)
    for t in args:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    return res


def _wants_f32(dtype):
    if dtype is torch.bfloat16:
        return False
    if dtype is torch.float32:
        return True
    raise ValueError("out_dtype must be bfloat16 or float32")


def moe_block_norm(x, residual=None, w_post=None, gate=None, w_pre=None, eps=1e-6, residual_scale=1.0,
                   block_scale=1.0, w_offset=0.0, quantize=False, res_out=None, h_out=None, stream=None):
    """r' = block_scale * gate * norm(x; w_post) + residual_scale * residual and h = norm(r'; w_pre).

    x, residual bf16 [M,H]; w_post, w_pre bf16 [H], each optional; gate bf16 [H] (per channel), fp32 [M] or
    [M,1] (per token) or bf16 [M,H].  Returns (r', h), h None without w_pre; with quantize=True
    (r', h, codes int8 [M,H], scales fp32 [M]).  Without residual, gate, w_post and block_scale, r' would be a copy
    of x: it is then only written where res_out asks for it, and returned as None otherwise.
    res_out and h_out may be x or residual itself."""
    if stream is not None:
        return _on(stream, _ops.block_norm, x, residual, w_post, gate, w_pre, eps, residual_scale, block_scale, w_offset,
                   quantize, res_out, h_out)
    return _ops.block_norm(x, residual, w_post, gate, w_pre, eps, residual_scale, block_scale, w_offset, quantize,
                           res_out, h_out)


def moe_int8_quantize(x, swiglu=False, stream=None):
    """(codes int8 [M,K], scales fp32 [M]) of the rows of x bf16 [M,K], or, swiglu=True, of clamp-SwiGLU of
    x = [gate | up] bf16 [M,2K]."""
    if stream is not None:
        return _on(stream, _ops.int8_quantize, x, swiglu)
    return _ops.int8_quantize(x, swiglu)


def moe_int8_gemm(q, q_s, w_q, w_s, add=None, out=None, out_dtype=torch.bfloat16, status_out=None, stream=None):
    """q_s[m] * w_s[n] * sum_c q[m,c] w_q[n,c] (+ add): q int8 [M,K], q_s fp32 [M], w_q int8 [N,K], w_s fp32 [N],
    add bf16 [M,N] -> [M,N] in out_dtype (bf16 or fp32).  A bf16 out may be add itself."""
    f32 = _wants_f32(out_dtype)
    if stream is not None:
        return _on(stream, _ops.int8_gemm, q, q_s, w_q, w_s, add, out, f32, status_out)
    return _ops.int8_gemm(q, q_s, w_q, w_s, add, out, f32, status_out)


def moe_grouped_gemm(x, w, expert_offsets, sorted_ids=None, k=1, swiglu=False, out=None, out_dtype=torch.bfloat16,
                     status_out=None, stream=None):
    """y[p] = w[e(p)] x[row(p)] over the expert-grouped order, or its clamp-SwiGLU.

    w bf16 [E,N,K] (swiglu=True: [E,2N,K], gate rows then up rows); expert_offsets int32 [E+1].  With sorted_ids
    int32 [M*k] (moe_permute's), x is bf16 [M,K] and row(p) = sorted_ids[p] // k; without, x is bf16 [R,K] in
    grouped order.  -> [R,N] in out_dtype (bf16 or fp32); positions that no expert's range holds keep what
    `out` held."""
    f32 = _wants_f32(out_dtype)
    if stream is not None:
        return _on(stream, _ops.grouped_gemm, x, w, expert_offsets, sorted_ids, k, swiglu, out, f32, status_out)
    return _ops.grouped_gemm(x, w, expert_offsets, sorted_ids, k, swiglu, out, f32, status_out)


def moe_combine(y, topk_w, inv_pos, add=None, out=None, stream=None):
    """out[t] = sum_j topk_w[t,j] * y[inv_pos[t*k+j]] (+ add[t]), bf16 [M,H]: y bf16 or fp32 [M*k,H] in expert-grouped
    order, topk_w fp32 [M,k], inv_pos int32 [M*k] (moe_permute's).  out may be add itself."""
    if stream is not None:
        return _on(stream, _ops.combine, y, topk_w, inv_pos, add, out)
    return _ops.combine(y, topk_w, inv_pos, add, out)
