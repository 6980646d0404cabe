"""Binding of the operators around the routed layer (include/moe.h, same names): the norms and residual
of the decoder block, int8 products for its shared expert, bf16 experts grouped by the routing.

Argument marshalling only.  All tensors of a call are on one CUDA device, which need not be the current
one; the work is enqueued on that device's current stream, or on `stream`, in which case outputs are
allocated for that stream and inputs are recorded on it.  A small call is over on the GPU in two or three
microseconds, so the way there is kept short: one pass over the arguments, no copies, no workspace."""
from __future__ import annotations

import torch

from ._lib import MoEError, load

_BF16, _F32, _I8, _I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32
_empty, _empty_like = torch.empty, torch.empty_like
_current_device, _raw_stream = torch.cuda.current_device, torch._C._cuda_getCurrentRawStream
_lib = load()

GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3


def _bad(name, t, dtype, shape, dev):
    if not isinstance(t, torch.Tensor):
        return TypeError("%s must be a tensor" % name)
    return ValueError("%s must be a contiguous %s tensor of shape %s on %s, got %s %s on %s%s" % (
        name, dtype, list(shape), "a CUDA device" if dev is None else "cuda:%d" % dev, t.dtype, list(t.shape), t.device,
        "" if t.is_contiguous() else " (strided)"))


def _ptr(name, t, dtype, shape, dev):
    """Address of t after checking type, shape, device and contiguity."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev \
            or not t.is_contiguous():
        raise _bad(name, t, dtype, shape, dev)
    return t.data_ptr()


def _lead(name, t, dtype, dims):
    """Index of the device the call runs on: t's."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.dim() != dims or not t.is_cuda \
            or not t.is_contiguous():
        raise _bad(name, t, dtype, ("?",) * dims, None)
    return t.get_device()


def _switched(fn, dev, stream, tensors, args):
    """fn on another device or stream: its outputs come from that stream's pool, its tensors are recorded on it."""
    if stream is None:
        with torch.cuda.device(dev):
            return fn(*args)
    if stream.device.index != dev:
        raise ValueError("stream is on %s, the tensors are on cuda:%d" % (stream.device, dev))
    with torch.cuda.stream(stream):
        res = fn(*args)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return res


def moe_block_norm(x, residual=None, w_post=None, gate=None, w_pre=None, eps=1e-6, residual_scale=1.0,
                   block_scale=1.0, w_offset=0.0, quantize=False, res_out=None, h_out=None, stream=None):
    """r' = block_scale * gate * norm(x; w_post) + residual_scale * residual and h = norm(r'; w_pre).

    x, residual bf16 [M,H]; w_post, w_pre bf16 [H], each optional; gate bf16 [H] (per channel), fp32 [M] or
    [M,1] (per token) or bf16 [M,H].  Returns (r', h), h None without w_pre; with quantize=True
    (r', h, codes int8 [M,H], scales fp32 [M]).  Without residual, gate, w_post and block_scale, r' would be a copy
    of x: it is then only written where res_out asks for it, and returned as None otherwise.
    res_out and h_out may be x or residual itself."""
    dev = _lead("x", x, _BF16, 2)
    if stream is not None or dev != _current_device():
        return _switched(moe_block_norm, dev, stream, (x, residual, w_post, gate, w_pre, res_out, h_out),
                         (x, residual, w_post, gate, w_pre, eps, residual_scale, block_scale, w_offset, quantize,
                          res_out, h_out))
    rows = x.shape
    M, H = rows
    rp = pp = np_ = gp = op = hp = q = qs = qp = sp = None
    kind = GATE_NONE
    if residual is not None:
        rp = _ptr("residual", residual, _BF16, rows, dev)
    if w_post is not None:
        pp = _ptr("w_post", w_post, _BF16, (H,), dev)
    if gate is not None:
        if not isinstance(gate, torch.Tensor):
            raise _bad("gate", gate, _BF16, (H,), dev)
        if gate.dtype is _F32:
            kind, gp = GATE_TOKEN, _ptr("gate", gate, _F32, (M, 1) if gate.dim() == 2 else (M,), dev)
        elif gate.dim() == 1:
            kind, gp = GATE_CHANNEL, _ptr("gate", gate, _BF16, (H,), dev)
        else:
            kind, gp = GATE_FULL, _ptr("gate", gate, _BF16, rows, dev)
    if res_out is not None:
        op = _ptr("res_out", res_out, _BF16, rows, dev)
    elif rp is not None or pp is not None or gp is not None or w_pre is None or block_scale != 1.0:
        res_out = _empty_like(x)
        op = res_out.data_ptr()
    if w_pre is not None:
        np_ = _ptr("w_pre", w_pre, _BF16, (H,), dev)
        if h_out is None:
            h_out = _empty_like(x)
            hp = h_out.data_ptr()
        else:
            hp = _ptr("h_out", h_out, _BF16, rows, dev)
    elif quantize or h_out is not None:
        raise ValueError("h and its codes need w_pre")
    if quantize:
        q, qs = _empty(M, H, dtype=_I8, device=x.device), _empty(M, dtype=_F32, device=x.device)
        qp, sp = q.data_ptr(), qs.data_ptr()
    rc = _lib.moe_block_norm(x.data_ptr(), rp, pp, gp, kind, np_, block_scale, residual_scale, eps, w_offset, op, hp, qp,
                             sp, M, H, _raw_stream(dev))
    if rc:
        raise MoEError(rc, "moe_block_norm")
    return (res_out, h_out, q, qs) if quantize else (res_out, h_out)


def moe_int8_quantize(x, swiglu=False, stream=None):
    """(codes int8 [M,K], scales fp32 [M]) of the rows of x bf16 [M,K], or, swiglu=True, of clamp-SwiGLU of
    x = [gate | up] bf16 [M,2K]."""
    dev = _lead("x", x, _BF16, 2)
    if stream is not None or dev != _current_device():
        return _switched(moe_int8_quantize, dev, stream, (x,), (x, swiglu))
    M, K = x.shape
    if swiglu:
        if K % 2:
            raise ValueError("x must hold as many gate as up columns, got %d in all" % K)
        K //= 2
    q, s = _empty(M, K, dtype=_I8, device=x.device), _empty(M, dtype=_F32, device=x.device)
    rc = _lib.moe_int8_quantize(x.data_ptr(), 1 if swiglu else 0, q.data_ptr(), s.data_ptr(), M, K, _raw_stream(dev))
    if rc:
        raise MoEError(rc, "moe_int8_quantize")
    return q, s


def moe_int8_gemm(q, q_s, w_q, w_s, add=None, out=None, out_dtype=torch.bfloat16, status_out=None, stream=None):
    """q_s[m] * w_s[n] * sum_c q[m,c] w_q[n,c] (+ add): q int8 [M,K], q_s fp32 [M], w_q int8 [N,K], w_s fp32 [N],
    add bf16 [M,N] -> [M,N] in out_dtype (bf16 or fp32).  A bf16 out may be add itself."""
    dev = _lead("q", q, _I8, 2)
    if stream is not None or dev != _current_device():
        return _switched(moe_int8_gemm, dev, stream, (q, q_s, w_q, w_s, add, out, status_out),
                         (q, q_s, w_q, w_s, add, out, out_dtype, status_out))
    M, K = q.shape
    if not isinstance(w_q, torch.Tensor) or w_q.dim() != 2:
        raise _bad("w_q", w_q, _I8, ("N", K), dev)
    N = w_q.shape[0]
    wp = _ptr("w_q", w_q, _I8, (N, K), dev)
    sp, cp = _ptr("q_s", q_s, _F32, (M,), dev), _ptr("w_s", w_s, _F32, (N,), dev)
    ap = None if add is None else _ptr("add", add, _BF16, (M, N), dev)
    tp = None if status_out is None else _ptr("status_out", status_out, _I32, (1,), dev)
    f32 = _wants_f32(out_dtype)
    if out is None:
        out = _empty(M, N, dtype=out_dtype, device=q.device)
        op = out.data_ptr()
    else:
        op = _ptr("out", out, out_dtype, (M, N), dev)
    rc = _lib.moe_int8_gemm(q.data_ptr(), sp, wp, cp, ap, op, f32, M, N, K, tp, _raw_stream(dev))
    if rc:
        raise MoEError(rc, "moe_int8_gemm")
    return out


def _wants_f32(dtype):
    if dtype is _BF16:
        return 0
    if dtype is _F32:
        return 1
    raise ValueError("out_dtype must be bfloat16 or float32")


def moe_grouped_gemm(x, w, expert_offsets, sorted_ids=None, k=1, swiglu=False, out=None, out_dtype=torch.bfloat16,
                     status_out=None, stream=None):
    """y[p] = w[e(p)] x[row(p)] over the expert-grouped order, or its clamp-SwiGLU.

    w bf16 [E,N,K] (swiglu=True: [E,2N,K], gate rows then up rows); expert_offsets int32 [E+1].  With sorted_ids
    int32 [M*k] (moe_permute's), x is bf16 [M,K] and row(p) = sorted_ids[p] // k; without, x is bf16 [R,K] in
    grouped order.  -> [R,N] in out_dtype (bf16 or fp32); positions that no expert's range holds keep what
    `out` held."""
    dev = _lead("x", x, _BF16, 2)
    if stream is not None or dev != _current_device():
        return _switched(moe_grouped_gemm, dev, stream, (x, w, expert_offsets, sorted_ids, out, status_out),
                         (x, w, expert_offsets, sorted_ids, k, swiglu, out, out_dtype, status_out))
    M, K = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise _bad("w", w, _BF16, ("E", "N", K), dev)
    E, N, _ = w.shape
    wp = _ptr("w", w, _BF16, (E, N, K), dev)
    if swiglu:
        if N % 2:
            raise ValueError("w must hold as many gate as up rows, got %d in all" % N)
        N //= 2
    fp = _ptr("expert_offsets", expert_offsets, _I32, (E + 1,), dev)
    tp = None if status_out is None else _ptr("status_out", status_out, _I32, (1,), dev)
    if sorted_ids is None:
        ip, k = None, 1
    else:
        if k < 1:
            raise ValueError("k must be at least 1")
        ip = _ptr("sorted_ids", sorted_ids, _I32, (M * k,), dev)
    f32 = _wants_f32(out_dtype)
    if out is None:
        out = _empty(M * k, N, dtype=out_dtype, device=x.device)
        op = out.data_ptr()
    else:
        op = _ptr("out", out, out_dtype, (M * k, N), dev)
    rc = _lib.moe_grouped_gemm(x.data_ptr(), wp, fp, ip, op, f32, 1 if swiglu else 0, M, N, K, E, k, tp,
                               _raw_stream(dev))
    if rc:
        raise MoEError(rc, "moe_grouped_gemm")
    return out


def moe_combine(y, topk_w, inv_pos, add=None, out=None, stream=None):
    """out[t] = sum_j topk_w[t,j] * y[inv_pos[t*k+j]] (+ add[t]), bf16 [M,H]: y bf16 or fp32 [M*k,H] in expert-grouped
    order, topk_w fp32 [M,k], inv_pos int32 [M*k] (moe_permute's).  out may be add itself."""
    f32 = isinstance(y, torch.Tensor) and y.dtype is _F32
    dev = _lead("y", y, _F32 if f32 else _BF16, 2)
    if stream is not None or dev != _current_device():
        return _switched(moe_combine, dev, stream, (y, topk_w, inv_pos, add, out), (y, topk_w, inv_pos, add, out))
    if not isinstance(topk_w, torch.Tensor) or topk_w.dim() != 2:
        raise _bad("topk_w", topk_w, _F32, ("M", "k"), dev)
    M, k = topk_w.shape
    R, H = y.shape
    if R != M * k:
        raise _bad("y", y, y.dtype, (M * k, H), dev)
    wp = _ptr("topk_w", topk_w, _F32, (M, k), dev)
    ip = _ptr("inv_pos", inv_pos, _I32, (R,), dev)
    ap = None if add is None else _ptr("add", add, _BF16, (M, H), dev)
    if out is None:
        out = _empty(M, H, dtype=_BF16, device=y.device)
        op = out.data_ptr()
    else:
        op = _ptr("out", out, _BF16, (M, H), dev)
    rc = _lib.moe_combine(y.data_ptr(), 1 if f32 else 0, wp, ip, ap, op, M, H, k, _raw_stream(dev))
    if rc:
        raise MoEError(rc, "moe_combine")
    return out
