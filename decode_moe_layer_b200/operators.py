"""Binding of the operators around the routed layer (include/moe.h, same names): the norms and residual
of the decoder block, int8 products for its shared expert, bf16 experts grouped by the routing.

Argument marshalling only.  All tensors of a call are on one CUDA device, which need not be the current
one; the work is enqueued on that device's current stream, or on `stream`, in which case outputs are
allocated for that stream and inputs are recorded on it."""
from __future__ import annotations

import torch

from ._lib import _check, load

_BF16, _F32, _I8, _I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32

GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3


def _bad(name, t, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        return TypeError("%s must be a tensor" % name)
    what = "x".join("?" if s is None else str(s) for s in shape)
    return ValueError("%s must be a contiguous %s tensor of shape [%s] on %s, got %s %s on %s%s" % (
        name, dtype, what, device, t.dtype, list(t.shape), t.device, "" if t.is_contiguous() else " (strided)"))


def _want(name, t, dtype, shape, device):
    """t as a pointer, after checking type, shape (None: any extent), device and contiguity."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != device or not t.is_contiguous() \
            or t.dim() != len(shape):
        raise _bad(name, t, dtype, shape, device)
    for have, want in zip(t.shape, shape):
        if want is not None and have != want:
            raise _bad(name, t, dtype, shape, device)
    return t.data_ptr()


def _lead(name, t, dtype, dims=2):
    """The tensor whose device the call runs on."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or not t.is_cuda or t.dim() != dims \
            or not t.is_contiguous():
        raise _bad(name, t, dtype, (None,) * dims, "a CUDA device")
    return t.device


def _out(name, t, dtype, shape, device):
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    return t, _want(name, t, dtype, shape, device)


def _elsewhere(device, stream):
    """Whether the call has to switch device or stream first."""
    return stream is not None or device.index != torch.cuda.current_device()


def _switched(fn, device, stream, tensors, args, kwargs):
    """fn on another device or stream: its outputs come from that stream's pool, its inputs are recorded."""
    if stream is None:
        with torch.cuda.device(device):
            return fn(*args, **kwargs)
    if stream.device != device:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, device))
    with torch.cuda.stream(stream):
        res = fn(*args, **kwargs)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return res


def _here(device):
    return torch._C._cuda_getCurrentRawStream(device.index)


def moe_block_norm(x, residual=None, w_post=None, gate=None, w_pre=None, eps=1e-6, residual_scale=1.0,
                   block_scale=1.0, w_offset=0.0, quantize=False, res_out=None, h_out=None, stream=None):
    """r' = block_scale * gate * norm(x; w_post) + residual_scale * residual and h = norm(r'; w_pre).

    x, residual bf16 [M,H]; w_post, w_pre bf16 [H], each optional; gate bf16 [H] (per channel), fp32 [M] or
    [M,1] (per token) or bf16 [M,H].  Returns (r', h), h None without w_pre; with quantize=True
    (r', h, codes int8 [M,H], scales fp32 [M]).  Without residual, gate and w_post, r' would be a copy of x:
    it is then only written where res_out asks for it, and returned as None otherwise.
    res_out and h_out may be x or residual itself."""
    dev = _lead("x", x, _BF16)
    if _elsewhere(dev, stream):
        return _switched(moe_block_norm, dev, stream, (x, residual, w_post, gate, w_pre, res_out, h_out),
                         (x, residual, w_post, gate, w_pre, eps, residual_scale, block_scale, w_offset, quantize,
                          res_out, h_out), {})
    M, H = x.shape
    rp = None if residual is None else _want("residual", residual, _BF16, (M, H), dev)
    pp = None if w_post is None else _want("w_post", w_post, _BF16, (H,), dev)
    np_ = None if w_pre is None else _want("w_pre", w_pre, _BF16, (H,), dev)
    if gate is None:
        kind, gp = GATE_NONE, None
    elif gate.dtype is _F32:
        kind, gp = GATE_TOKEN, _want("gate", gate, _F32, (M, 1) if gate.dim() == 2 else (M,), dev)
    elif gate.dim() == 1:
        kind, gp = GATE_CHANNEL, _want("gate", gate, _BF16, (H,), dev)
    else:
        kind, gp = GATE_FULL, _want("gate", gate, _BF16, (M, H), dev)
    if w_pre is None and (quantize or h_out is not None):
        raise ValueError("h and its codes need w_pre")
    op = hp = q = qs = qp = sp = None
    if res_out is not None or residual is not None or gate is not None or w_post is not None or w_pre is None:
        res_out, op = _out("res_out", res_out, _BF16, (M, H), dev)
    if w_pre is not None:
        h_out, hp = _out("h_out", h_out, _BF16, (M, H), dev)
    if quantize:
        q, qp = _out("q", None, _I8, (M, H), dev)
        qs, sp = _out("q_s", None, _F32, (M,), dev)
    _check(load().moe_block_norm(x.data_ptr(), rp, pp, gp, kind, np_, block_scale, residual_scale, eps, w_offset, op,
                                 hp, qp, sp, M, H, _here(dev)), "moe_block_norm")
    return (res_out, h_out, q, qs) if quantize else (res_out, h_out)


def moe_int8_quantize(x, swiglu=False, stream=None):
    """(codes int8 [M,K], scales fp32 [M]) of the rows of x bf16 [M,K], or, swiglu=True, of clamp-SwiGLU of
    x = [gate | up] bf16 [M,2K]."""
    dev = _lead("x", x, _BF16)
    if _elsewhere(dev, stream):
        return _switched(moe_int8_quantize, dev, stream, (x,), (x, swiglu), {})
    M, K = x.shape
    if swiglu:
        if K % 2:
            raise ValueError("x must hold as many gate as up columns, got %d in all" % K)
        K //= 2
    q = torch.empty((M, K), dtype=_I8, device=dev)
    s = torch.empty((M,), dtype=_F32, device=dev)
    _check(load().moe_int8_quantize(x.data_ptr(), 1 if swiglu else 0, q.data_ptr(), s.data_ptr(), M, K, _here(dev)),
           "moe_int8_quantize")
    return q, s


def moe_int8_gemm(q, q_s, w_q, w_s, add=None, out=None, out_dtype=torch.bfloat16, status_out=None, stream=None):
    """q_s[m] * w_s[n] * sum_c q[m,c] w_q[n,c] (+ add): q int8 [M,K], q_s fp32 [M], w_q int8 [N,K], w_s fp32 [N],
    add bf16 [M,N] -> [M,N] in out_dtype (bf16 or fp32).  A bf16 out may be add itself."""
    dev = _lead("q", q, _I8)
    if _elsewhere(dev, stream):
        return _switched(moe_int8_gemm, dev, stream, (q, q_s, w_q, w_s, add, out, status_out),
                         (q, q_s, w_q, w_s, add, out, out_dtype, status_out), {})
    if out_dtype is not _BF16 and out_dtype is not _F32:
        raise ValueError("out_dtype must be bfloat16 or float32")
    M, K = q.shape
    wp = _want("w_q", w_q, _I8, (None, K), dev)
    N = w_q.shape[0]
    ap = None if add is None else _want("add", add, _BF16, (M, N), dev)
    tp = None if status_out is None else _want("status_out", status_out, _I32, (1,), dev)
    sp, cp = _want("q_s", q_s, _F32, (M,), dev), _want("w_s", w_s, _F32, (N,), dev)
    out, op = _out("out", out, out_dtype, (M, N), dev)
    _check(load().moe_int8_gemm(q.data_ptr(), sp, wp, cp, ap, op, 1 if out_dtype is _F32 else 0, M, N, K, tp,
                                _here(dev)), "moe_int8_gemm")
    return out


def moe_grouped_gemm(x, w, expert_offsets, sorted_ids=None, k=1, swiglu=False, out=None, out_dtype=torch.bfloat16,
                     status_out=None, stream=None):
    """y[p] = w[e(p)] x[row(p)] over the expert-grouped order, or its clamp-SwiGLU.

    w bf16 [E,N,K] (swiglu=True: [E,2N,K], gate rows then up rows); expert_offsets int32 [E+1].  With sorted_ids
    int32 [M*k] (moe_permute's), x is bf16 [M,K] and row(p) = sorted_ids[p] // k; without, x is bf16 [R,K] in
    grouped order.  -> [R,N] in out_dtype (bf16 or fp32); positions that no expert's range holds keep what
    `out` held."""
    dev = _lead("x", x, _BF16)
    if _elsewhere(dev, stream):
        return _switched(moe_grouped_gemm, dev, stream, (x, w, expert_offsets, sorted_ids, out, status_out),
                         (x, w, expert_offsets, sorted_ids, k, swiglu, out, out_dtype, status_out), {})
    if out_dtype is not _BF16 and out_dtype is not _F32:
        raise ValueError("out_dtype must be bfloat16 or float32")
    M, K = x.shape
    wp = _want("w", w, _BF16, (None, None, K), dev)
    E, N, _ = w.shape
    if swiglu:
        if N % 2:
            raise ValueError("w must hold as many gate as up rows, got %d in all" % N)
        N //= 2
    fp = _want("expert_offsets", expert_offsets, _I32, (E + 1,), dev)
    tp = None if status_out is None else _want("status_out", status_out, _I32, (1,), dev)
    if sorted_ids is None:
        ip, k = None, 1
    else:
        if k < 1:
            raise ValueError("k must be at least 1")
        ip = _want("sorted_ids", sorted_ids, _I32, (M * k,), dev)
    out, op = _out("out", out, out_dtype, (M * k, N), dev)
    _check(load().moe_grouped_gemm(x.data_ptr(), wp, fp, ip, op, 1 if out_dtype is _F32 else 0, 1 if swiglu else 0, M,
                                   N, K, E, k, tp, _here(dev)), "moe_grouped_gemm")
    return out


def moe_combine(y, topk_w, inv_pos, add=None, out=None, stream=None):
    """out[t] = sum_j topk_w[t,j] * y[inv_pos[t*k+j]] (+ add[t]), bf16 [M,H]: y bf16 or fp32 [M*k,H] in expert-grouped
    order, topk_w fp32 [M,k], inv_pos int32 [M*k] (moe_permute's).  out may be add itself."""
    f32 = isinstance(y, torch.Tensor) and y.dtype is _F32
    dev = _lead("y", y, _F32 if f32 else _BF16)
    if _elsewhere(dev, stream):
        return _switched(moe_combine, dev, stream, (y, topk_w, inv_pos, add, out), (y, topk_w, inv_pos, add, out), {})
    wp = _want("topk_w", topk_w, _F32, (None, None), dev)
    M, k = topk_w.shape
    H = y.shape[1]
    if y.shape[0] != M * k:
        raise _bad("y", y, y.dtype, (M * k, H), dev)
    ip = _want("inv_pos", inv_pos, _I32, (M * k,), dev)
    ap = None if add is None else _want("add", add, _BF16, (M, H), dev)
    out, op = _out("out", out, _BF16, (M, H), dev)
    _check(load().moe_combine(y.data_ptr(), 1 if f32 else 0, wp, ip, ap, op, M, H, k, _here(dev)), "moe_combine")
    return out
