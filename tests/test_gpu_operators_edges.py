"""The operators around the routed layer where a value is no number, an index is wrong or a wait gives up: against plain
implementations in 64 bits, with the tolerances of test_gpu_operators.py where none is derived here."""
import pytest
import torch

from tests.test_gpu_operators import BF, D, F32, close, gen, int8_ref, ints, moe, quant_ref, randn  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

NAN = float("nan")


# ------------------------------------------------------------------ int8 codes

# a vector of 8 a thread (M <= 148 and K <= 8192) and four
@pytest.mark.parametrize("M,K", [(2, 16), (5, 2048), (3, 16384), (149, 768), (200, 8208)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_nan_reaches_the_scale_of_its_row(moe, M, K, swiglu):
    g = gen(M + K)
    x = randn(g, M, 2 * K if swiglu else K, scale=3.0)
    q0, s0 = moe.moe_int8_quantize(x, swiglu=swiglu)
    columns = [0, K // 2, K - 1] + ([K, 2 * K - 8] if swiglu else [])    # of swiglu: gate and up
    for i, c in enumerate(columns):
        bad, y = (i * 7 + 1) % M, x.clone()
        y[bad, c] = NAN if i % 2 else -NAN
        q, s = moe.moe_int8_quantize(y, swiglu=swiglu)
        keep = torch.arange(M, device="cuda") != bad
        assert torch.isnan(s[bad]) and (q[bad] == 0).all(), c
        assert torch.equal(s[keep], s0[keep]) and torch.equal(q[keep], q0[keep])
        # and, through the product, all of its row and no other
        n = 5
        w, ws = ints(g, -9, 9, n, K, dtype=torch.int8), torch.ones(n, device="cuda")
        for m in (slice(0, M), slice(bad, bad + 1)):      # in tiles (M > 4), by rows
            y8 = moe.moe_int8_gemm(q[m].contiguous(), s[m].contiguous(), w, ws)
            assert torch.isnan(y8[keep[m].logical_not()]).all() and torch.isfinite(y8[keep[m]]).all()


@pytest.mark.parametrize("M", [3, 160])
def test_inf_makes_an_infinite_scale_and_codes_of_zero(moe, M):
    x = randn(gen(M), M, 256)
    x[1, 17] = -float("inf")
    q, s = moe.moe_int8_quantize(x)
    assert s[1] == float("inf") and (q[1] == 0).all() and torch.isfinite(s[0]) and torch.isfinite(s[2:]).all()


@pytest.mark.parametrize("M,H", [(3, 512), (700, 512), (200, 4112)])
def test_norm_codes_of_a_nan_weight(moe, M, H):
    # the row's sum of squares is finite, one element of h is not
    g = gen(M)
    x, w = randn(g, M, H), randn(g, H)
    w[H - 3] = NAN
    _, h, q, s = moe.moe_block_norm(x, w_pre=w, quantize=True)
    assert torch.isnan(s).all() and (q == 0).all()
    assert torch.isnan(h[:, H - 3]).all() and torch.isfinite(h[:, :H - 3]).all()


# exp and the division within 2 units in the last place (2^-22) each, 1 + t, two products and the division by 127 half a
# unit (2^-24) each: 12 * 2^-24.  At -88 the value is still inside fp32's normal range.
@pytest.mark.parametrize("gate", [(-88.0, -88.0), (-88.5, -80.0), (-60.0, -20.0), (-20.0, -5.0), (-5.0, 10.0)])
@pytest.mark.parametrize("M,K", [(4, 64), (200, 512)])
def test_swiglu_codes_keep_fp32(moe, gate, M, K):
    g = gen(K)
    lo, hi = gate
    x = torch.cat([lo + (hi - lo) * torch.rand(M, K, generator=g, device="cuda"),
                   3 + 3 * torch.rand(M, K, generator=g, device="cuda")], 1).to(BF)
    q, s = moe.moe_int8_quantize(x, swiglu=True)
    a, u = x[:, :K].to(D).clamp(max=7), x[:, K:].to(D).clamp(-7, 7)
    v = a * torch.sigmoid(a) * u
    top = v.abs().amax(1)
    close(s, top / 127, 12 * 2.0 ** -24 * top / 127, "scale")
    # the code is the nearest of 127 v / max, each of v and max off by as much
    t = 127 * v / top[:, None]
    close(q, t, torch.full_like(t, 0.5 + 127 * 24 * 2.0 ** -24), "codes")


def test_codes_of_tiny_rows(moe):
    # down to bf16's smallest subnormals, where the row's scale has few bits left or none: 127 v / max all the same
    g = gen(3)
    x = torch.randn(64, 272, generator=g, device="cuda", dtype=F32)
    e = -90.0 - torch.arange(64, device="cuda") * 0.75             # rows of about 2^-90 .. 2^-137
    x = (x.to(D) * 2.0 ** e.to(D)[:, None]).to(BF)
    x[:, 1] = x.abs().amax(1)                                      # ties: the code 63.5 (where bf16 holds the half)
    x[:, 2] = x[:, 1] / 2
    q, s = moe.moe_int8_quantize(x)
    rq, rs = quant_ref(x.float().cpu())
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu(), rq), "rows %s" % (q.cpu() != rq).any(1).nonzero().flatten().tolist()


# ------------------------------------------------------------------ grouped products: wrong and empty groups, odd rows

def clamped(off, R):
    """Group starts as moe.h has them for wrong offsets: inside 0..R and ascending."""
    return torch.cummax(off.long().clamp(0, R), 0).values.tolist()


def fill_ref(y, x, w, off, ids, k):
    R, o = y.shape[0], clamped(off, y.shape[0])
    for e in range(len(o) - 1):
        lo, hi = o[e], o[e + 1]
        if lo < hi:
            rows = (ids[lo:hi].long() % 2 ** 32 // k).clamp(max=x.shape[0] - 1) if ids is not None else slice(lo, hi)
            y[lo:hi] = (x[rows].to(D) @ w[e].to(D).T).to(F32).to(y.dtype)
    return y


# R, E: by rows (R <= 2/3 E, or 16 rows at most in no more groups), in tiles
GROUPS = [(12, 64), (12, 12), (300, 900), (40, 8), (700, 8)]


@pytest.mark.parametrize("R,E", GROUPS)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("wrong", ["descending", "negative", "beyond", "late", "random"])
def test_wrong_offsets_leave_right_groups_right(moe, R, E, gather, wrong):
    g = gen(R * 3 + E)
    N, K, k = 36, 200, 2
    x, w = ints(g, -4, 4, R // k if gather else R, K), ints(g, -4, 4, E, N, K)
    off = torch.randint(0, R + 1, (E + 1,), generator=g, device="cuda").sort().values
    off[0], off[E] = 0, R
    if wrong == "descending":
        off[1], off[2] = 5, 4
        off[E // 2:E // 2 + 3] = off[E // 2:E // 2 + 3].flip(0)
    elif wrong == "negative":
        off[0], off[1], off[E // 2] = -3, -2 ** 31, -1
    elif wrong == "beyond":
        off[E - 1], off[E] = R + 1, 2 ** 31 - 1
    elif wrong == "late":
        off[:3] = torch.tensor([4, 2, 5], device="cuda")
        off[E] = R - 3
    else:
        off = torch.randint(-R, 2 * R, (E + 1,), generator=g, device="cuda")
    off = off.int()
    ids = torch.randperm(R, generator=g, device="cuda").int() if gather else None
    if gather:
        ids[[0, R // 2]] = torch.tensor([-7, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    guard = torch.full((R + 64, N), 5.0, device="cuda", dtype=BF)
    moe.moe_grouped_gemm(x, w, off, ids, k=k, out=guard[:R])
    assert (guard[R:] == 5).all()
    assert torch.equal(guard[:R], fill_ref(torch.full((R, N), 5.0, device="cuda", dtype=BF), x, w, off, ids, k))


@pytest.mark.parametrize("R,E", GROUPS)
@pytest.mark.parametrize("swiglu", [False, True])
def test_rows_outside_the_groups_stay_either_way(moe, R, E, swiglu):
    g = gen(R + E)
    N, K = 20, 136
    x, w = ints(g, -4, 4, R, K), ints(g, -4, 4, E, 2 * N if swiglu else N, K)
    off = (5 + (torch.rand(E + 1, generator=g, device="cuda") * (R - 8)).long().sort().values).clamp(max=R - 3).int()
    for o in (off, torch.zeros_like(off), torch.full_like(off, R)):
        for dt in (BF, F32):
            y = torch.full((R, N), 77.0, dtype=dt, device="cuda")
            moe.moe_grouped_gemm(x, w, o, out=y, out_dtype=dt, swiglu=swiglu)
            live = torch.zeros(R, dtype=torch.bool, device="cuda")
            live[int(o[0]):int(o[E])] = True
            assert (y[~live] == 77).all()
            if not swiglu:
                assert torch.equal(y, fill_ref(torch.full_like(y, 77.0), x, w, o, None, 1))
            else:
                assert (y[live].abs() <= 49).all()


@pytest.mark.parametrize("R,E", GROUPS)
@pytest.mark.parametrize("K", [8, 200, 520])
def test_nan_rows_stay_in_their_rows_either_way(moe, R, E, K):
    g = gen(R + K)
    N = 33
    x, w = ints(g, -4, 4, R, K), ints(g, -4, 4, E, N, K)
    off = torch.randint(0, R + 1, (E + 1,), generator=g, device="cuda").sort().values.int()
    off[0], off[E] = 0, R
    ref = moe.moe_grouped_gemm(x, w, off, out_dtype=F32)
    bad = torch.zeros(R, dtype=torch.bool, device="cuda")
    bad[[1, R // 2, R - 1]] = True
    x[bad] = NAN
    y = moe.moe_grouped_gemm(x, w, off, out_dtype=F32)
    assert torch.equal(y[~bad], ref[~bad]) and torch.isnan(y[bad]).all()


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("N", [1, 2, 3, 5, 127, 1001])
@pytest.mark.parametrize("K", [16, 272, 4112])
def test_int8_gemm_of_few_rows_and_odd_columns(moe, M, N, K):
    g = gen(M * 17 + N + K)
    q, w = ints(g, -128, 127, M, K, dtype=torch.int8), ints(g, -128, 127, N, K, dtype=torch.int8)
    qs, ws = torch.rand(M, generator=g, device="cuda") + 0.5, torch.rand(N, generator=g, device="cuda") + 0.5
    guard = torch.full((M * N + 64,), 5.0, device="cuda")
    y = moe.moe_int8_gemm(q, qs, w, ws, out=guard[:M * N].view(M, N), out_dtype=F32)
    ref = int8_ref(q, qs, w, ws)
    close(y, ref, 4 * 2.0 ** -24 * ref.abs() + 1e-30)
    assert (guard[M * N:] == 5).all()


# ------------------------------------------------------------------ waits that give up

# 16 and 4 stages' worth of rows a CTA, one row a CTA, rows of one and of several vectors a thread
@pytest.mark.parametrize("M,H", [(592, 64), (1500, 1024), (700, 8), (20000, 264), (160, 8192), (1000, 16384)])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("quantize", [False, True])
def test_norm_rows_whose_copies_do_not_come_are_nan(moe, M, H, post, quantize):
    g = gen(M + H)
    x, r, w = randn(g, M, H), randn(g, M, H), randn(g, H)
    ref = moe.moe_block_norm(x, residual=r, w_post=w if post else None, w_pre=w, quantize=True)
    out = [torch.zeros_like(t) for t in ref]
    moe.moe_selftest_norm_timeout(x, r, w if post else None, w, out[0], out[1], out[2] if quantize else None,
                                  out[3] if quantize else None)
    torch.cuda.synchronize()
    lost = torch.isnan(out[0]).all(1)
    assert lost[0] and not lost.all()
    assert torch.isnan(out[1][lost]).all()
    rows = lost.nonzero().flatten()
    if rows.numel() > 1:
        step = int(rows[1])
        assert step >= 148 and torch.equal(rows, torch.arange(0, M, step, device="cuda"))     # one CTA's
    assert torch.equal(out[0][~lost], ref[0][~lost]) and torch.equal(out[1][~lost], ref[1][~lost])
    if quantize:
        assert torch.isnan(out[3][lost]).all() and (out[2][lost] == 0).all()
        assert torch.equal(out[2][~lost], ref[2][~lost]) and torch.equal(out[3][~lost], ref[3][~lost])
    again = moe.moe_block_norm(x, residual=r, w_post=w if post else None, w_pre=w, quantize=True)
    assert all(torch.equal(a, b) for a, b in zip(again, ref))


def lost_and_right(y, ref, status):
    """Mask of the NaN of y, once all else is what it should be."""
    assert status.item() == -5
    lost = torch.isnan(y)
    assert torch.equal(y[~lost], ref[~lost]) and lost.any() and not lost.all()
    return lost


# one tile a cluster, with K cut among two and four pairs and not; several tiles a cluster, the last in halves
@pytest.mark.parametrize("M,N,K,once", [(33, 1536, 2048, True), (128, 1536, 2048, True), (40, 1000, 8192, True), (6, 700, 4096, True),
                                        (256, 4096, 7168, True), (64, 520, 144, True), (200, 1024, 768, True),
                                        (2500, 4096, 400, False), (1500, 4100, 2000, False)])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_int8_tiles_whose_copies_do_not_come_are_nan(moe, M, N, K, once, out_dtype):
    g = gen(M + N + K)
    q, w = ints(g, -128, 127, M, K, dtype=torch.int8), ints(g, -128, 127, N, K, dtype=torch.int8)
    qs, ws = torch.rand(M, generator=g, device="cuda") + 0.5, torch.rand(N, generator=g, device="cuda") + 0.5
    ref = moe.moe_int8_gemm(q, qs, w, ws, out_dtype=out_dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full_like(ref, 3.0)
    moe.moe_selftest_product_timeout(q, w, y, status, q_s=qs, w_s=ws)
    lost = lost_and_right(y, ref, status)
    assert lost[0, :256].all()
    if once:      # a tile of 256 columns, whole
        assert (lost[:, :256] == lost[:, :1]).all() and not lost[:, 256:].any()
    z = moe.moe_int8_gemm(q, qs, w, ws, out_dtype=out_dtype, status_out=status)
    assert status.item() == 0 and torch.equal(z, ref)


@pytest.mark.parametrize("cuts,N,K", [([3, 20, 20, 60], 768, 2048), ([0, 40, 48, 100], 600, 4096), ([2, 300, 700, 701, 1200], 4096, 136),
                                      ([0, 90], 1024, 4096), ([0, 129, 258, 387, 516, 3000], 1024, 136)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_tiles_whose_copies_do_not_come_are_nan(moe, cuts, N, K, gather, swiglu):
    R, E = cuts[-1] + 5, len(cuts) - 1
    g = gen(R + N)
    x, w = randn(g, R, K), randn(g, E, 2 * N if swiglu else N, K, scale=K ** -0.5)
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    ids = torch.randperm(R, generator=g, device="cuda").int() if gather else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dt in (BF, F32):
        ref = moe.moe_grouped_gemm(x, w, off, ids, swiglu=swiglu, out=torch.full((R, N), 7.0, dtype=dt, device="cuda"),
                                   out_dtype=dt)
        y = torch.full((R, N), 7.0, dtype=dt, device="cuda")
        moe.moe_selftest_product_timeout(x, w, y, status, expert_offsets=off, sorted_ids=ids, swiglu=swiglu)
        lost = lost_and_right(y, ref, status)
        first = 128 if swiglu else 256
        assert lost[cuts[0], :first].all()
        assert (lost[:, :first] == lost[:, :1]).all()
        z = moe.moe_grouped_gemm(x, w, off, ids, swiglu=swiglu, out=y.fill_(7), out_dtype=dt, status_out=status)
        assert status.item() == 0 and torch.equal(z, ref)


# ------------------------------------------------------------------ in place

@pytest.mark.parametrize("M,H", [(700, 1024), (160, 8192), (3000, 264)])     # rows through the ring of copies
@pytest.mark.parametrize("gate", [False, True])
def test_norm_in_place_of_many_rows(moe, M, H, gate):
    g = gen(M + 1)
    x, r, w = randn(g, M, H), randn(g, M, H), randn(g, H)
    kw = dict(w_post=w, w_pre=w, gate=randn(g, M, H) if gate else None, quantize=True)
    ref = moe.moe_block_norm(x, residual=r, **kw)
    for swap in (False, True):
        a, b = x.clone(), r.clone()
        got = moe.moe_block_norm(a, residual=b, res_out=a if swap else b, h_out=b if swap else a, **kw)
        assert got[0] is (a if swap else b) and all(torch.equal(u, v) for u, v in zip(got, ref))
