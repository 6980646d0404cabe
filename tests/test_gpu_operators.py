"""The operators around the routed layer against plain implementations in 64 bits.

Tolerances, per element:
  * rounding to the output: 2^-8 |ref| for bf16 (half a step), 2^-24 |ref| for fp32;
  * a bf16 product of length K: K additions in fp32 of at most the sum of magnitudes S, each off by at
    most 2^-23 of it (the tensor cores need not round to nearest), so K 2^-23 S, and 8 more for the joined parts;
    products and sums of small integers are exact in fp32 and are compared for equality;
  * an int8 product: the sum is exact; its conversion, two scalings and one addition are 4 roundings of fp32;
  * a norm: a sum of squares is 26 additions deep at most, then a division, a root (2 ulp) and under ten
    products: below 64 roundings of fp32, 2^-18 of the magnitudes added;
  * SwiGLU: |d silu| <= 1.1 |dg| and |silu| <= 7, |u| <= 7, so an error d of g and u gives at most 15 d, and expf and
    the division a few ulp of the result (2^-20 of it).
"""
import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

D = torch.float64
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    import decode_moe_layer_b200 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def ints(g, lo, hi, *shape, dtype=BF):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(dtype)


def close(got, ref, tol, what=""):
    err = (got.to(D) - ref).abs()
    assert torch.isfinite(got).all(), what + ": not finite"
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, "%s: %.3f of the tolerance" % (what, worst)


# ------------------------------------------------------------------ block norm

def norm_ref(x, residual, w_post, gate, w_pre, eps, rs, bs, off):
    z = x.to(D)
    if w_post is not None:
        z = z / torch.sqrt((z * z).mean(1, keepdim=True) + eps) * (w_post.to(D) + off)
    if gate is not None:
        z = z * (gate.to(D).reshape(-1, 1) if gate.dtype == F32 else gate.to(D))
    z = z * bs
    r, mag = z, z.abs()
    if residual is not None:
        r = z + rs * residual.to(D)
        mag = mag + (rs * residual.to(D)).abs()
    if w_pre is None:
        return r, mag, None, None
    f = (w_pre.to(D) + off) / torch.sqrt((r * r).mean(1, keepdim=True) + eps)
    return r, mag, r * f, mag * f.abs()


@pytest.mark.parametrize("M,H", [(1, 8), (1, 7168), (3, 264), (5, 1000), (33, 2048), (2, 8192), (2, 8200), (7, 16384),
                                 (700, 512), (600, 4104), (593, 16384), (1500, 1024), (148, 4104), (149, 4104),
                                 (149, 4096), (200, 7168), (149, 16384)])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post,res,pre", [(True, True, True), (False, True, True), (True, False, True),
                                          (True, True, False), (False, False, True)])
def test_block_norm(moe, M, H, gate, post, res, pre):
    g = gen(M * 131 + H)
    x, r = randn(g, M, H, scale=0.7), randn(g, M, H, scale=2.0) if res else None
    wp = randn(g, H, scale=0.2) if post else None
    wn = randn(g, H, scale=0.2) if pre else None
    gt = {"none": None, "channel": randn(g, H), "token": torch.rand(M, generator=g, device="cuda"),
          "full": randn(g, M, H)}[gate]
    quant = pre and H % 16 == 0
    got = moe.moe_block_norm(x, residual=r, w_post=wp, gate=gt, w_pre=wn, eps=1e-5, residual_scale=0.875,
                             block_scale=1.25, w_offset=1.0, quantize=quant)
    rr, mag, hh, hmag = norm_ref(x, r, wp, gt, wn, 1e-5, 0.875, 1.25, 1.0)
    if got[0] is None:
        assert not res and not post and gate == "none"
    else:
        close(got[0], rr, 2.0 ** -8 * rr.abs() + 2.0 ** -18 * mag + 1e-30, "r'")
    if not pre:
        assert got[1] is None
        return
    close(got[1], hh, 2.0 ** -8 * hh.abs() + 2.0 ** -18 * hmag + 1e-30, "h")
    if quant:
        q, s = got[2], got[3]
        top = hh.abs().amax(1)
        close(s, top / 127, 2.0 ** -17 * hmag.amax(1) / 127 + 1e-30, "scale")
        # half a step of the code, and what the scale and h are off by
        half = 0.5 * s.to(D)[:, None]
        close(q.to(D) * s.to(D)[:, None], hh, half + 2.0 ** -16 * hmag.amax(1, keepdim=True) + 1e-30, "codes")
        assert q.abs().max().item() <= 127
        assert ((q.abs() == 127).any(1) | (s == 0)).all()


def test_block_norm_in_place_and_plain(moe):
    g = gen(5)
    x, r, w = randn(g, 17, 1024), randn(g, 17, 1024), randn(g, 1024)
    a, b = moe.moe_block_norm(x, residual=r, w_post=w, w_pre=w)
    x2, r2 = x.clone(), r.clone()
    c, d = moe.moe_block_norm(x2, residual=r2, w_post=w, w_pre=w, res_out=r2, h_out=x2)
    assert c is r2 and d is x2 and torch.equal(a, r2) and torch.equal(b, x2)
    n, h = moe.moe_block_norm(x, w_pre=w)
    assert n is None and h.shape == x.shape
    y = torch.empty_like(x)
    n, h2 = moe.moe_block_norm(x, w_pre=w, res_out=y)
    assert torch.equal(y, x) and torch.equal(h, h2)


@pytest.mark.parametrize("M,H", [(1, 264), (3, 1000), (31, 8192), (32, 8192), (33, 8192), (64, 16384), (0, 64)])
def test_outputs_of_a_call_do_not_meet(moe, M, H):
    # up to 1 MB two outputs share an allocation, beyond each has its own
    g = gen(M + H)
    x, r, w = randn(g, M, H), randn(g, M, H), randn(g, H)
    quant = H % 16 == 0
    outs = moe.moe_block_norm(x, residual=r, w_pre=w, quantize=quant)
    outs += moe.moe_int8_quantize(x) if quant else ()
    for i, t in enumerate(outs):
        assert t.is_contiguous() and t.data_ptr() % 16 == 0
        assert t.shape == ((M,) if t.dtype == F32 else (M, H))
        others = [o.clone() for o in outs]
        if t.numel() > 0:
            assert t.storage_offset() * t.element_size() + t.numel() * t.element_size() <= t.untyped_storage().nbytes()
        keep = t.clone()
        t.fill_(17)
        for j, o in enumerate(outs):
            assert j == i or torch.equal(o, others[j])
        t.copy_(keep)
    small = 0 < (M * H * 2 + 511) // 512 * 512 + M * H * 2 <= 1 << 20
    assert (outs[0].untyped_storage().data_ptr() == outs[1].untyped_storage().data_ptr()) == (small or M == 0)
    # one output alone is not kept from its place by the other's
    a = outs[0].clone()
    h = moe.moe_block_norm(x, residual=r, w_pre=w, res_out=outs[0])[1]
    assert torch.equal(a, outs[0]) and torch.equal(h, outs[1])


def test_block_norm_token_gate_as_column(moe):
    g = gen(8)
    x, r, w = randn(g, 9, 640), randn(g, 9, 640), randn(g, 640)
    t = torch.rand(9, generator=g, device="cuda")
    a = moe.moe_block_norm(x, residual=r, gate=t, w_pre=w)
    b = moe.moe_block_norm(x, residual=r, gate=t[:, None].contiguous(), w_pre=w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_block_norm_zero_rows_and_nan_rows(moe):
    g = gen(6)
    x, r, w = randn(g, 6, 512), randn(g, 6, 512), randn(g, 512)
    x[2] = 0
    r[2] = 0
    x[4, 100] = float("nan")
    res, h, q, s = moe.moe_block_norm(x, residual=r, w_post=w, w_pre=w, quantize=True)
    assert (res[2] == 0).all() and (h[2] == 0).all() and (q[2] == 0).all() and s[2] == 0
    assert torch.isnan(h[4].float()).all()
    keep = [0, 1, 2, 3, 5]
    ref = moe.moe_block_norm(x[keep].contiguous(), residual=r[keep].contiguous(), w_post=w, w_pre=w)
    assert torch.equal(ref[0], res[keep]) and torch.equal(ref[1], h[keep])


# ------------------------------------------------------------------ int8

def quant_ref(v):
    """Codes and scales as the definition gives them: 127 v is exact in 64 bits and a tie's quotient too."""
    top = v.abs().amax(1)
    q = torch.where(top[:, None] > 0, 127 * v.to(D) / top[:, None].to(D), torch.zeros_like(v, dtype=D))
    return torch.round(q).to(torch.int8), top / np.float32(127)


def test_int8_codes_of_ties(moe):
    # every bf16 mantissa as a row's largest value: its half has the code 63.5, which goes to the even neighbour whatever
    # the rounding of the scale; 2 max / 254 * odd is a tie too where bf16 holds it
    top = (torch.arange(128, 256, device="cuda") * 2.0 ** -3).to(BF)
    x = torch.zeros(128, 64, dtype=BF, device="cuda")
    x[:, 0], x[:, 1], x[:, 2] = top, top / 2, -top / 2
    x[126, 3:35] = (torch.arange(32, device="cuda") * 2 + 1).to(BF) * 2.0 ** -3   # of 254 / 8: codes n + 1/2
    q, _ = moe.moe_int8_quantize(x)
    assert (q[:, 0] == 127).all() and (q[:, 1] == 64).all() and (q[:, 2] == -64).all()
    want = torch.round(torch.arange(32, device="cuda", dtype=D) + 0.5).to(torch.int8)
    assert torch.equal(q[126, 3:35], want)
    h = moe.moe_block_norm(x, w_pre=torch.ones(64, dtype=BF, device="cuda"), quantize=True)
    assert (h[2][:, 1] == -h[2][:, 2]).all() and ((h[2][:, 1] == 63) | (h[2][:, 1] == 64)).all()


@pytest.mark.parametrize("M,K", [(1, 16), (1, 7168), (3, 272), (33, 2048), (5, 8208), (2, 16384), (600, 768)])
def test_int8_quantize(moe, M, K):
    g = gen(K)
    x = randn(g, M, K, scale=3.0)
    x[0] *= 2.0 ** -60
    if M > 1:
        x[1] = 0
    q, s = moe.moe_int8_quantize(x)
    rq, rs = quant_ref(x.float().cpu())
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)


@pytest.mark.parametrize("M,K", [(1, 16), (2, 768), (33, 2048), (3, 16384)])
def test_int8_quantize_swiglu(moe, M, K):
    g = gen(K + 1)
    x = randn(g, M, 2 * K, scale=5.0)
    q, s = moe.moe_int8_quantize(x, swiglu=True)
    a, u = x[:, :K].to(D).clamp(max=7), x[:, K:].to(D).clamp(-7, 7)
    v = a * torch.sigmoid(a) * u
    top = v.abs().amax(1)
    close(s, top / 127, 2.0 ** -19 * top / 127)
    close(q.to(D) * s.to(D)[:, None], v, 0.5 * s.to(D)[:, None] + 2.0 ** -18 * top[:, None])


def int8_ref(q, qs, w, ws):
    return (q.to(D) @ w.to(D).T) * qs.to(D)[:, None] * ws.to(D)[None, :]


INT8_SHAPES = [(1, 8, 16), (1, 1, 16), (1, 4096, 7168), (2, 1000, 528), (16, 128, 128), (17, 129, 144), (31, 512, 2048),
               (33, 1536, 2048), (64, 256, 4096), (65, 200, 1040), (100, 640, 512), (129, 96, 256), (200, 1024, 768),
               (256, 128, 1024), (257, 384, 2048), (513, 2056, 400), (1000, 4096, 1536),
               (40, 1000, 8192), (100, 4096, 7168), (200, 1500, 4112), (6, 200, 65536), (2100, 2700, 272), (1500, 4100, 2000), (5000, 1000, 1024)]


@pytest.mark.parametrize("M,N,K", INT8_SHAPES)
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("with_add", [False, True])
def test_int8_gemm(moe, M, N, K, out_dtype, with_add):
    g = gen(M + N + K)
    q, w = ints(g, -128, 127, M, K, dtype=torch.int8), ints(g, -128, 127, N, K, dtype=torch.int8)
    qs, ws = torch.rand(M, generator=g, device="cuda") + 0.5, (torch.rand(N, generator=g, device="cuda") + 0.5) * 1e-4
    add = randn(g, M, N, scale=50.0) if with_add else None
    status = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    y = moe.moe_int8_gemm(q, qs, w, ws, add=add, out_dtype=out_dtype, status_out=status)
    prod = int8_ref(q, qs, w, ws)
    ref = prod + (add.to(D) if with_add else 0)
    mag = prod.abs() + (add.to(D).abs() if with_add else 0)
    half = 2.0 ** -8 if out_dtype == BF else 2.0 ** -24
    assert status.item() == 0
    close(y, ref, half * ref.abs() + 4 * 2.0 ** -24 * mag + 1e-30)
    if with_add and out_dtype == BF:
        z = moe.moe_int8_gemm(q, qs, w, ws, add=add, out=add)
        assert z is add and torch.equal(z, y)


def test_int8_gemm_largest_sums(moe):
    # every product at its largest magnitude: the int32 sum is exact and far outside 24 bits
    K = 65536
    q = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((130, K), -128, dtype=torch.int8, device="cuda")
    w[7] = 127
    one = torch.ones(130, device="cuda")
    y = moe.moe_int8_gemm(q, one[:3], w, one, out_dtype=F32)
    ref = torch.full((3, 130), 128.0 * 128 * K, dtype=D, device="cuda")
    ref[:, 7] = -128.0 * 127 * K
    assert torch.equal(y.to(D), ref)


# Calls of more tiles than CTA pairs (74) whose last wave is less than half full: its tiles run as two halves each.
@pytest.mark.parametrize("M,N", [(2500, 4096), (2354, 4096), (2560, 4000), (1100, 8192), (4096, 4096), (20000, 512)])
def test_int8_gemm_last_wave(moe, M, N):
    g = gen(M + N)
    K = 400
    q, w = ints(g, -128, 127, M, K, dtype=torch.int8), ints(g, -128, 127, N, K, dtype=torch.int8)
    one = torch.ones(max(M, N), device="cuda")
    y = moe.moe_int8_gemm(q, one[:M], w, one[:N], out_dtype=F32)
    assert torch.equal(y.to(D), q.to(D) @ w.to(D).T)     # sums below 2^24: exact in fp32


@pytest.mark.parametrize("cuts,N", [([0, 300, 300, 812, 1200], 4096), ([0, 1100], 8192), ([7, 250, 2600, 2600, 2616], 4096),
                                    ([0, 129, 258, 387, 516, 3000], 2048), ([0, 20, 700, 740, 996, 996], 5000)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_gemm_last_wave(moe, cuts, N, gather, swiglu):
    R, E, K = cuts[-1] + 9, len(cuts) - 1, 136
    g = gen(R + N + E)
    if swiglu:
        N //= 2
    x, w = ints(g, -4, 4, R, K), ints(g, -4, 4, E, 2 * N if swiglu else N, K)
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    ids = torch.randperm(R, generator=g, device="cuda").int() if gather else None
    out = torch.full((R, N), 5.0, device="cuda")
    y = moe.moe_grouped_gemm(x, w, off, ids, k=1, swiglu=swiglu, out=out, out_dtype=F32)
    assert (y[:cuts[0]] == 5).all() and (y[cuts[-1]:] == 5).all()
    for e in range(E):
        lo, hi = cuts[e], cuts[e + 1]
        p = (x[ids[lo:hi].long()] if gather else x[lo:hi]).to(D) @ w[e].to(D).T
        if not swiglu:
            assert torch.equal(y[lo:hi].to(D), p)
            continue
        a, u = p[:, :N].clamp(max=7), p[:, N:].clamp(-7, 7)
        ref = a * torch.sigmoid(a) * u
        # the sums are exact; exp, the division and two products are off by a few units of 2^-24 each, exp's argument is
        # at most 16 K, but where it is large and negative the value is below 2^-100
        close(y[lo:hi], ref, 2.0 ** -20 * ref.abs() + 2.0 ** -100, "group %d" % e)


# ------------------------------------------------------------------ grouped

def grouping(g, M, k, E, how):
    """(offsets, sorted_ids, inv_pos, ids) of M*k assignments."""
    R = M * k
    if how == "uniform":
        ids = torch.rand(M, E, generator=g, device="cuda").topk(k, 1).indices.reshape(-1)
    elif how == "one":                                # everything on the last expert
        ids = torch.full((R,), E - 1, device="cuda")
    else:                                             # skew: most rows on a few, many experts empty
        u = torch.rand(R, generator=g, device="cuda")
        ids = (E * u ** 4).long().clamp(max=E - 1)
    order = torch.sort(ids, stable=True).indices
    off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    off[1:] = torch.bincount(ids, minlength=E).cumsum(0)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(R, device="cuda")
    return off.int(), order.int(), inv.int(), ids


def grouped_ref(x, w, off, ids, k, swiglu):
    """y and the magnitude sums, in 64 bits."""
    off = off.tolist()
    R = off[-1]
    N = w.shape[1]
    y = torch.zeros(R, N, dtype=D, device="cuda")
    m = torch.zeros(R, N, dtype=D, device="cuda")
    for e in range(len(off) - 1):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        xe = (x[ids[lo:hi].long() // k] if ids is not None else x[lo:hi]).to(D)
        y[lo:hi] = xe @ w[e].to(D).T
        m[lo:hi] = xe.abs() @ w[e].to(D).abs().T
    if not swiglu:
        return y, m
    N //= 2
    a, u = y[:, :N].clamp(max=7), y[:, N:].clamp(-7, 7)
    return a * torch.sigmoid(a) * u, torch.maximum(m[:, :N], m[:, N:])


GROUPED_SHAPES = [
    # M, k, E, N, K, how
    (1, 1, 1, 16, 8, "uniform"), (1, 8, 128, 768, 2048, "uniform"), (1, 4, 16, 512, 1024, "uniform"),
    (2, 4, 16, 512, 1024, "uniform"), (8, 8, 128, 768, 2048, "uniform"), (3, 2, 60, 144, 72, "uniform"),
    (5, 3, 7, 1040, 1000, "skew"), (64, 4, 16, 256, 512, "uniform"), (64, 4, 16, 256, 512, "one"),
    (200, 2, 8, 384, 264, "skew"), (300, 4, 1000, 128, 256, "skew"), (257, 1, 3, 272, 520, "skew"),
    (129, 8, 8, 160, 136, "skew"), (700, 8, 16, 512, 1024, "uniform"), (1024, 8, 128, 256, 1536, "skew"),
    (513, 4, 2, 1024, 2048, "skew"), (1500, 2, 3, 1296, 200, "skew"), (700, 8, 32, 1536, 520, "uniform"),
    (640, 8, 100, 1024, 1024, "skew"), (5000, 1, 1, 528, 1032, "uniform"),
    (40, 2, 3, 520, 4096, "skew"), (300, 1, 2, 130, 8192, "skew"), (20, 1, 1, 1000, 4104, "uniform"),
    (600, 2, 2, 200, 4096, "skew"), (33, 2, 5, 77, 64, "uniform"), (5, 3, 7, 1001, 1000, "skew"), (2000, 1, 2, 2051, 136, "skew"),
]


@pytest.mark.parametrize("M,k,E,N,K,how", GROUPED_SHAPES)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_gemm(moe, M, k, E, N, K, how, gather, swiglu):
    g = gen(M * 7 + N + K)
    off, ids, _, _ = grouping(g, M, k, E, how)
    x = randn(g, M if gather else M * k, K)
    w = randn(g, E, 2 * N if swiglu else N, K, scale=2.0 / K ** 0.5)
    status = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    ref, mag = grouped_ref(x, w, off, ids if gather else None, k, swiglu)
    acc = (K + 8) * 2.0 ** -23 * mag
    for dt, half in ((BF, 2.0 ** -8), (F32, 2.0 ** -24)):
        y = moe.moe_grouped_gemm(x, w, off, ids if gather else None, k=k, swiglu=swiglu, out_dtype=dt,
                                 status_out=status)
        assert status.item() == 0 and y.dtype == dt
        tol = half * ref.abs() + ((15 * acc + 2.0 ** -20 * ref.abs()) if swiglu else acc) + 1e-30
        close(y, ref, tol, str(dt))
        rel = ((y.to(D) - ref).norm() / ref.norm()).item()
        assert rel <= (2.0 ** -8 if dt == BF else 2.0 ** -16), rel


@pytest.mark.parametrize("M,k,E,N,K,how", GROUPED_SHAPES)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_gemm_exact_on_integers(moe, M, k, E, N, K, how, gather):
    # |sum| <= 16 K < 2^24: every partial sum is an fp32 number whatever the order
    g = gen(M + N)
    off, ids, _, _ = grouping(g, M, k, E, how)
    x, w = ints(g, -4, 4, M if gather else M * k, K), ints(g, -4, 4, E, N, K)
    ref, _ = grouped_ref(x, w, off, ids if gather else None, k, False)
    y = moe.moe_grouped_gemm(x, w, off, ids if gather else None, k=k, out_dtype=F32)
    assert torch.equal(y.to(D), ref)
    y = moe.moe_grouped_gemm(x, w, off, ids if gather else None, k=k)
    assert torch.equal(y, ref.to(F32).to(BF))


@pytest.mark.parametrize("R,k,E,N,K", [(102, 2, 52, 2883, 1960), (60, 4, 43, 1995, 1576), (700, 2, 40, 1230, 664)])
def test_gather_of_tiny_and_larger_groups_in_turn(moe, R, k, E, N, K):
    # groups of less than 17 rows leave warps of the gather without rows; they have to keep in step all the same
    g = gen(R + E)
    off, ids, _, _ = grouping(g, R // k, k, E, "skew" if R == 700 else "uniform")
    x, w = ints(g, -4, 4, R // k, K), ints(g, -4, 4, E, N, K)
    ref, _ = grouped_ref(x, w, off, ids, k, False)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(30):
        y = moe.moe_grouped_gemm(x, w, off, ids, k=k, out_dtype=F32, status_out=status)
        assert status.item() == 0 and torch.equal(y.to(D), ref)


@pytest.mark.parametrize("R,E,nt_hint", [(40, 8, "narrow"), (3000, 8, "wide")])
def test_grouped_rows_outside_the_groups_stay(moe, R, E, nt_hint):
    g = gen(R)
    N, K = 160, 256
    x, w = ints(g, -4, 4, R, K), ints(g, -4, 4, E, N, K)
    # the first group starts at 5, the last ends 7 before the end, two in the middle are empty
    cuts = torch.linspace(5, R - 7, E - 1).long()
    off = torch.cat([cuts[:3], cuts[2:3], cuts[2:3], cuts[3:]]).int().cuda()
    assert off.numel() == E + 1
    for dt in (BF, F32):
        y = torch.full((R, N), 77.0, dtype=dt, device="cuda")
        moe.moe_grouped_gemm(x, w, off, out=y, out_dtype=dt)
        o = off.tolist()
        ref = torch.full((R, N), 77.0, dtype=D, device="cuda")
        for e in range(E):
            ref[o[e]:o[e + 1]] = x[o[e]:o[e + 1]].to(D) @ w[e].to(D).T
        assert torch.equal(y, ref.to(F32).to(dt))


def test_grouped_all_groups_empty(moe):
    x, w = torch.ones(4, 64, device="cuda", dtype=BF), torch.ones(3, 32, 64, device="cuda", dtype=BF)
    y = torch.full((4, 32), 3.0, device="cuda", dtype=BF)
    moe.moe_grouped_gemm(x, w, torch.zeros(4, dtype=torch.int32, device="cuda"), out=y)
    assert (y == 3).all()
    assert moe.moe_grouped_gemm(x[:0], w, torch.zeros(4, dtype=torch.int32, device="cuda")).shape == (0, 32)


def test_grouped_nan_rows_stay_in_their_rows(moe):
    # a bad row, and bad rows next to a group's end, inside the same token tile
    g = gen(9)
    R, E, N, K = 50, 4, 96, 192
    x, w = ints(g, -4, 4, R, K), ints(g, -4, 4, E, N, K)
    off = torch.tensor([0, 3, 20, 21, 50], dtype=torch.int32, device="cuda")
    ref = moe.moe_grouped_gemm(x, w, off, out_dtype=F32)
    bad = [3, 20, 49]
    x[bad] = float("nan")
    x[3] = float("inf")
    y = moe.moe_grouped_gemm(x, w, off, out_dtype=F32)
    good = [i for i in range(R) if i not in bad]
    assert torch.equal(y[good], ref[good]) and not torch.isfinite(y[bad]).any()


def test_grouped_bad_indices_stay_inside(moe):
    # offsets and ids outside their ranges are clamped: nothing is read or written outside the tensors, and the
    # groups that are right come out right
    g = gen(10)
    M, k, E, N, K = 6, 2, 4, 64, 128
    x, w = ints(g, -4, 4, M, K), ints(g, -4, 4, E, N, K)
    off = torch.tensor([0, 5, 4, 9, 100000], dtype=torch.int32, device="cuda")   # descending, then beyond the end
    ids = torch.tensor([0, 3, 5, -7, 11, 2, 900, 1, 4, 6, 8, 10], dtype=torch.int32, device="cuda")
    guard = torch.full((M * k + 64, N), 5.0, device="cuda", dtype=BF)
    y = guard[:M * k]
    moe.moe_grouped_gemm(x, w, off, ids, k=k, out=y)
    assert (guard[M * k:] == 5).all()
    rows = torch.tensor([0, 1, 2], device="cuda")
    ref = x[rows].to(D) @ w[0].to(D).T
    assert torch.equal(y[:3], ref.to(F32).to(BF))


def test_grouped_no_dependence_on_timing(moe):
    g = gen(11)
    off, ids, _, _ = grouping(g, 8, 8, 128, "uniform")
    x, w = randn(g, 8, 2048), randn(g, 128, 768, 2048, scale=0.05)
    a = moe.moe_grouped_gemm(x, w, off, ids, k=8, out_dtype=F32)
    for _ in range(5):
        assert torch.equal(a, moe.moe_grouped_gemm(x, w, off, ids, k=8, out_dtype=F32))


# ------------------------------------------------------------------ combine

@pytest.mark.parametrize("M,k,H", [(1, 1, 8), (1, 8, 2048), (3, 6, 1000), (33, 8, 7168), (5, 32, 520), (700, 4, 512)])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("with_add", [False, True])
def test_combine(moe, M, k, H, dt, with_add):
    g = gen(M + H)
    y = randn(g, M * k, H, dtype=dt)
    w = torch.softmax(torch.randn(M, k, generator=g, device="cuda"), 1)
    inv = torch.randperm(M * k, generator=g, device="cuda").int()
    if M > 1:
        inv[3] = -1                # dropped
        inv[4] = M * k
        inv[k] = inv[0]            # the same row twice
    add = randn(g, M, H) if with_add else None
    out = moe.moe_combine(y, w, inv, add=add)
    pos = inv.long()
    ok = (pos >= 0) & (pos < M * k)
    rows = torch.where(ok[:, None], y.to(D)[pos.clamp(0, M * k - 1)], torch.zeros((), dtype=D, device="cuda"))
    rows = (rows * w.to(D).reshape(-1, 1)).view(M, k, H)
    ref, mag = rows.sum(1), rows.abs().sum(1)
    if with_add:
        ref, mag = ref + add.to(D), mag + add.to(D).abs()
    close(out, ref, 2.0 ** -8 * ref.abs() + (k + 1) * 2.0 ** -24 * mag + 1e-30)
    if with_add:
        z = moe.moe_combine(y, w, inv, add=add, out=add)
        assert z is add and torch.equal(z, out)


# ------------------------------------------------------------------ together

def _block(moe, t, k):
    """A decoder block's second half: norm, routed bf16 experts beside an int8 shared expert, norm and residual."""
    r1, h, q, qs = moe.moe_block_norm(t["attn"], residual=t["res"], w_post=t["n1"], w_pre=t["n2"], quantize=True)
    ids, tw = moe.moe_route(h, t["router"], k)
    E = t["router"].shape[0]
    off, srt, inv = moe.moe_permute(ids, E)
    hh = moe.moe_grouped_gemm(h, t["w13"], off, srt, k=k, swiglu=True)
    yy = moe.moe_grouped_gemm(hh, t["w2"], off)
    gu = moe.moe_int8_gemm(q, qs, t["s13"], t["s13s"])
    q2, q2s = moe.moe_int8_quantize(gu, swiglu=True)
    shared = moe.moe_int8_gemm(q2, q2s, t["s2"], t["s2s"])
    out = moe.moe_combine(yy, tw, inv, add=shared)
    r2, n = moe.moe_block_norm(out, residual=r1, w_post=t["n1"], gate=t["gate"], w_pre=t["n2"])
    return r1, h, q, qs, ids, tw, off, srt, inv, hh, yy, gu, q2, q2s, out, r2, n


def _block_inputs(M, H, I, E, seed):
    g = gen(seed)
    t = {"attn": randn(g, M, H), "res": randn(g, M, H), "n1": 1 + randn(g, H, scale=0.1),
         "n2": 1 + randn(g, H, scale=0.1), "gate": randn(g, H), "router": randn(g, E, H, scale=H ** -0.5, dtype=F32),
         "w13": randn(g, E, 2 * I, H, scale=H ** -0.5), "w2": randn(g, E, H, I, scale=I ** -0.5),
         "s13": ints(g, -100, 100, 2 * I, H, dtype=torch.int8), "s2": ints(g, -100, 100, H, I, dtype=torch.int8)}
    t["s13s"] = torch.rand(2 * I, generator=g, device="cuda") * 0.02 * H ** -0.5
    t["s2s"] = torch.rand(H, generator=g, device="cuda") * 0.02 * I ** -0.5
    return t


@pytest.mark.parametrize("M", [1, 9, 130])
def test_block_of_all_of_them(moe, M):
    H, I, E, k = 1024, 512, 16, 4
    t = _block_inputs(M, H, I, E, M)
    r1, h, q, qs, ids, tw, off, srt, inv, hh, yy, gu, q2, q2s, out, r2, n = _block(moe, t, k)
    # each step from the step's own stored inputs, in 64 bits
    rr, mag, hr, hm = norm_ref(t["attn"], t["res"], t["n1"], None, t["n2"], 1e-6, 1.0, 1.0, 0.0)
    close(r1, rr, 2.0 ** -8 * rr.abs() + 2.0 ** -18 * mag)
    close(h, hr, 2.0 ** -8 * hr.abs() + 2.0 ** -18 * hm)
    ref, m = grouped_ref(h, t["w13"], off, srt, k, True)
    close(hh, ref, 2.0 ** -8 * ref.abs() + 15 * (H + 8) * 2.0 ** -23 * m + 2.0 ** -20)
    ref, m = grouped_ref(hh, t["w2"], off, None, 1, False)
    close(yy, ref, 2.0 ** -8 * ref.abs() + (I + 8) * 2.0 ** -23 * m)
    ref = int8_ref(q, qs, t["s13"], t["s13s"])
    close(gu, ref, (2.0 ** -8 + 2.0 ** -22) * ref.abs() + 1e-30)
    shared = int8_ref(q2, q2s, t["s2"], t["s2s"])
    flat = torch.arange(M * k, device="cuda")
    assert torch.equal(srt[inv.long()].long(), flat)
    routed = (yy.to(D)[inv.long()].view(M, k, H) * tw.to(D)[:, :, None])
    ref, m = routed.sum(1) + shared, routed.abs().sum(1) + shared.abs()
    close(out, ref, 2.0 ** -8 * (ref.abs() + shared.abs()) + (k + 5) * 2.0 ** -24 * m)
    rr, mag, hr, hm = norm_ref(out, r1, t["n1"], t["gate"], t["n2"], 1e-6, 1.0, 1.0, 0.0)
    close(r2, rr, 2.0 ** -8 * rr.abs() + 2.0 ** -18 * mag)
    close(n, hr, 2.0 ** -8 * hr.abs() + 2.0 ** -18 * hm)


def test_shared_expert_beside_the_mxfp4_layer(moe):
    # the library's routed MXFP4 layer between the norms, its output taken into the shared expert's product
    from moe_inputs import generator as mg
    from tests import _gpu_util as U
    inp = mg.make_inputs(0, 2)
    d = U.device_inputs(inp)
    H, I = inp.shape.H, inp.shape.I
    t = _block_inputs(2, H, I, 2, 77)
    x = U.bits_to_bf16_tensor(inp.x)
    r1, h, q, qs = moe.moe_block_norm(x, residual=t["res"], w_pre=t["n2"], quantize=True)
    routed = moe.moe_mxfp4_forward(h, d["router_w"], d["w13_q"], d["w13_s"], d["w2_q"], d["w2_s"], inp.shape.k)
    keep = routed.clone()
    q2, q2s = moe.moe_int8_quantize(moe.moe_int8_gemm(q, qs, t["s13"], t["s13s"]), swiglu=True)
    out = moe.moe_int8_gemm(q2, q2s, t["s2"], t["s2s"], add=routed, out=routed)
    ref = int8_ref(q2, q2s, t["s2"], t["s2s"])
    mag = ref.abs() + keep.to(D).abs()
    ref = ref + keep.to(D)
    close(out, ref, 2.0 ** -8 * ref.abs() + 4 * 2.0 ** -24 * mag)


def test_block_captured_and_replayed_on_two_streams(moe):
    H, I, E, k = 1024, 512, 16, 4
    graphs, outs, refs, inputs = [], [], [], []
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    cap = torch.cuda.Stream()
    for i, M in enumerate((5, 40)):
        t = _block_inputs(M, H, I, E, 100 + i)
        inputs.append(t)
        with torch.cuda.stream(cap):
            _block_steps(moe, t, k, None)
        torch.cuda.synchronize()
        route = moe.moe_route(moe.moe_block_norm(t["attn"], residual=t["res"], w_post=t["n1"], w_pre=t["n2"])[1],
                              t["router"], k)
        inputs.append(route)                  # the graphs read them: they live as long
        refs.append(_block_steps(moe, t, k, route))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=cap):
            outs.append(_block_steps(moe, t, k, route))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(10):                       # both graphs at once: nothing is shared between them
        for s, g in zip(side, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, refs):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


def _block_steps(moe, t, k, route):
    """The new operators of _block alone (routing given), so that graphs share no library workspace."""
    r1, h, q, qs = moe.moe_block_norm(t["attn"], residual=t["res"], w_post=t["n1"], w_pre=t["n2"], quantize=True)
    if route is None:
        return (r1, h)
    ids, tw = route
    off, srt, inv = moe.moe_permute(ids, t["router"].shape[0])
    yy = moe.moe_grouped_gemm(moe.moe_grouped_gemm(h, t["w13"], off, srt, k=k, swiglu=True), t["w2"], off)
    q2, q2s = moe.moe_int8_quantize(moe.moe_int8_gemm(q, qs, t["s13"], t["s13s"]), swiglu=True)
    out = moe.moe_combine(yy, tw, inv, add=moe.moe_int8_gemm(q2, q2s, t["s2"], t["s2s"]))
    return moe.moe_block_norm(out, residual=r1, w_post=t["n1"], gate=t["gate"], w_pre=t["n2"])


def test_stream_argument(moe):
    g = gen(12)
    x, w = randn(g, 9, 2048), randn(g, 2048)
    ref = moe.moe_block_norm(x, w_pre=w)[1]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = moe.moe_block_norm(x, w_pre=w, stream=s)[1]
    s.synchronize()
    assert torch.equal(got, ref)
    q, qs = moe.moe_int8_quantize(x, stream=s)
    w8 = ints(g, -90, 90, 64, 2048, dtype=torch.int8)
    torch.cuda.synchronize()
    y = moe.moe_int8_gemm(q, qs, w8, w[:64].float(), stream=s)
    s.synchronize()
    assert torch.equal(y, moe.moe_int8_gemm(q, qs, w8, w[:64].float()))


def test_binding_refusals(moe):
    g = gen(13)
    x, w = randn(g, 4, 64), randn(g, 64)
    with pytest.raises(ValueError):
        moe.moe_block_norm(x.t(), w_pre=w)
    with pytest.raises(ValueError):
        moe.moe_block_norm(x, w_pre=w[:32])
    with pytest.raises(ValueError):
        moe.moe_block_norm(x, w_pre=w.cpu())
    with pytest.raises(ValueError):
        moe.moe_block_norm(x, quantize=True)
    with pytest.raises(ValueError):
        moe.moe_block_norm(x, residual=x[:3], w_pre=w)
    with pytest.raises(moe.MoEError):
        moe.moe_block_norm(x, w_pre=w, eps=0.0)
    with pytest.raises(ValueError):
        moe.moe_int8_quantize(x.float())
    with pytest.raises(moe.MoEError):
        moe.moe_int8_quantize(randn(g, 4, 24))
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, randn(g, 2, 16, 32), torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, randn(g, 2, 16, 64), torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_combine(x, torch.ones(2, 3, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda"))
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    w3 = randn(g, 2, 16, 64)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, w3.transpose(1, 2).contiguous().transpose(1, 2), z)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, w3, z.long())
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, w3, z, torch.zeros(9, dtype=torch.int32, device="cuda"), k=2)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, w3, z, torch.zeros(0, dtype=torch.int32, device="cuda"), k=0)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, w3[:, :15].contiguous(), z, swiglu=True)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, w3, z, out=torch.zeros(4, 16, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, w3, z, out_dtype=torch.float16)
    with pytest.raises(moe.MoEError):
        moe.moe_grouped_gemm(randn(g, 4, 20), randn(g, 2, 16, 20), z)
    with pytest.raises(TypeError):
        moe.moe_grouped_gemm(x, w3, None)
    with pytest.raises(ValueError):
        moe.moe_int8_gemm(*moe.moe_int8_quantize(x), torch.zeros(8, 32, dtype=torch.int8, device="cuda"), w[:8].float())
    with pytest.raises(ValueError):
        moe.moe_int8_quantize(x, stream=_FakeStream(torch.device("cuda", 1)))
    assert moe.moe_combine(x[:0], torch.ones(0, 3, device="cuda"), z[:0]).shape == (0, 64)
    assert moe.moe_block_norm(x[:0], w_pre=w)[1].shape == (0, 64)


class _FakeStream:
    def __init__(self, device):
        self.device = device


# ------------------------------------------------------------------ more than 2^31 elements

def _room(gib):
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip("needs %d GiB of device memory" % gib)


def test_outputs_beyond_32_bit_offsets(moe):
    _room(40)
    g = gen(20)
    # int8 product: 40000 x 60000 outputs
    M, N, K = 40000, 60000, 32
    q, w = ints(g, -9, 9, M, K, dtype=torch.int8), ints(g, -9, 9, N, K, dtype=torch.int8)
    one = torch.ones(max(M, N), device="cuda")
    y = moe.moe_int8_gemm(q, one[:M], w, one[:N])
    for rows in (slice(0, 3), slice(M - 300, M)):
        assert torch.equal(y[rows], (q[rows].to(D) @ w.to(D).T).to(F32).to(BF))
    del y
    # grouped: 300000 rows of 8192, three groups
    R, N, K = 300000, 8192, 64
    x, w = ints(g, -4, 4, R, K), ints(g, -4, 4, 3, N, K)
    off = torch.tensor([0, 5, 290000, R], dtype=torch.int32, device="cuda")
    y = moe.moe_grouped_gemm(x, w, off)
    for e, lo, hi in ((0, 0, 5), (1, 289500, 290000), (2, 290000, 290300), (2, R - 300, R)):
        assert torch.equal(y[lo:hi], (x[lo:hi].to(D) @ w[e].to(D).T).to(F32).to(BF))
    # combine takes those rows in reverse, two a token
    inv = torch.arange(R - 1, -1, -1, dtype=torch.int32, device="cuda")
    tw = torch.rand(R // 2, 2, generator=g, device="cuda")
    out = moe.moe_combine(y, tw, inv)
    t = torch.tensor([0, 1, R // 2 - 1], device="cuda")
    ref = sum(y[inv[2 * t + j].long()].to(D) * tw[t, j].to(D)[:, None] for j in range(2))
    mag = sum((y[inv[2 * t + j].long()].to(D) * tw[t, j].to(D)[:, None]).abs() for j in range(2))
    close(out[t], ref, 2.0 ** -8 * ref.abs() + 3 * 2.0 ** -24 * mag + 1e-30)
    del out
    # norm and codes of the same rows
    wn = randn(g, N)
    r, h = moe.moe_block_norm(y, residual=y, w_pre=wn)
    rows = slice(R - 200, R)
    r2, h2 = moe.moe_block_norm(y[rows].contiguous(), residual=y[rows].contiguous(), w_pre=wn)
    close(r[rows], r2.to(D), 2.0 ** -7 * r2.to(D).abs() + 1e-30)
    close(h[rows], h2.to(D), 2.0 ** -7 * h2.to(D).abs() + 2.0 ** -16)
    del r, h
    q, s = moe.moe_int8_quantize(y)
    rq, rs = quant_ref(y[rows].float().cpu())
    assert torch.equal(q[rows].cpu(), rq) and torch.equal(s[rows].cpu(), rs)


@pytest.mark.parametrize("M", [1, 40])
def test_weights_beyond_32_bit_offsets(moe, M):
    _room(20)
    g = gen(21)
    E, N, K, k = 40, 8192, 8192, 2
    w = torch.zeros(E, N, K, device="cuda", dtype=BF)
    w[E - 1] = ints(g, -4, 4, N, K)
    w[E - 2] = ints(g, -4, 4, N, K)
    x = ints(g, -4, 4, M, K)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E - 1] = M
    off[E] = 2 * M
    ids = torch.cat([torch.arange(M) * 2, torch.arange(M) * 2 + 1]).int().cuda()
    y = moe.moe_grouped_gemm(x, w, off, ids, k=k)
    assert torch.equal(y[:M], (x.to(D) @ w[E - 2].to(D).T).to(F32).to(BF))
    assert torch.equal(y[M:], (x.to(D) @ w[E - 1].to(D).T).to(F32).to(BF))
