"""Argument checks of the operators around the routed layer: the C entry points refuse before they make any CUDA
call, and the Python binding refuses tensors of the wrong type, shape, layout or device.  No GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import decode_moe_layer_b200 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
P = ctypes.c_void_p
INV, UNS, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE, moe.MOE_OK


def _norm(**kw):
    a = dict(x=0x100000, residual=0x200000, w_post=0x300000, gate=None, kind=0, w_pre=0x310000, b=1.0, r=1.0, eps=1e-6,
             off=0.0, res_out=0x400000, h_out=0x500000, q=None, qs=None, M=8, H=2048)
    a.update(kw)
    p = {n: None if a[n] is None else P(a[n]) for n in ("x", "residual", "w_post", "gate", "w_pre", "res_out", "h_out",
                                                       "q", "qs")}
    return moe.load().moe_block_norm(p["x"], p["residual"], p["w_post"], p["gate"], a["kind"], p["w_pre"], a["b"],
                                     a["r"], a["eps"], a["off"], p["res_out"], p["h_out"], p["q"], p["qs"], a["M"],
                                     a["H"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=0), OK), (dict(M=0, x=None, res_out=None), OK), (dict(M=-1), INV), (dict(H=0), INV), (dict(H=2044), UNS),
    (dict(H=16392), UNS), (dict(M=(1 << 22) + 1), UNS), (dict(x=None), INV), (dict(x=0x100008), INV),
    (dict(residual=0x200002), INV), (dict(eps=0.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV),
    (dict(b=float("inf")), INV), (dict(r=float("nan")), INV), (dict(off=float("nan")), INV), (dict(kind=4), INV),
    (dict(kind=-1), INV), (dict(kind=1), INV), (dict(gate=0x600000), INV), (dict(kind=2, gate=0x600002), INV),
    (dict(kind=1, gate=0x600004), INV), (dict(res_out=None, h_out=None, w_pre=None), INV), (dict(w_pre=None), INV),
    (dict(h_out=None), INV), (dict(q=0x700000), INV), (dict(qs=0x700000), INV), (dict(q=0x700008, qs=0x800000), INV),
    (dict(res_out=0x100010), INV), (dict(h_out=0x200010), INV), (dict(h_out=0x400000), INV),
    (dict(q=0x100000, qs=0x800000), INV), (dict(kind=3, gate=0x400000), INV), (dict(w_post=0x500010), INV),
])
def test_block_norm_refusals(kw, want):
    assert _norm(**kw) == want


def test_int8_refusals():
    lib = moe.load()

    def quant(x=0x100000, sw=0, q=0x200000, s=0x300000, M=8, K=2048):
        return lib.moe_int8_quantize(P(x) if x else None, sw, P(q) if q else None, P(s) if s else None, M, K, None)

    assert quant(M=0) == OK and quant(M=0, x=0) == OK
    assert quant(M=-1) == INV and quant(K=0) == INV and quant(x=0) == INV and quant(q=0) == INV and quant(s=0) == INV
    assert quant(K=2040) == UNS and quant(K=16400) == UNS
    assert quant(x=0x100008) == INV and quant(q=0x200004) == INV and quant(s=0x300001) == INV
    assert quant(q=0x100000 + 8 * 2048) == INV                      # codes inside x
    assert quant(q=0x100000 + 2 * 8 * 2048, sw=1) == INV            # inside x once x holds gate and up

    def gemm(q=0x100000, qs=0x200000, w=0x300000, ws=0x900000, add=0, out=0xA00000, f32=0, M=8, N=512, K=2048, st=0):
        n = lambda v: P(v) if v else None  # noqa: E731
        return lib.moe_int8_gemm(n(q), n(qs), n(w), n(ws), n(add), n(out), f32, M, N, K, n(st), None)

    assert gemm(M=0) == OK and gemm(M=0, q=0, out=0) == OK
    assert gemm(M=-1) == INV and gemm(N=0) == INV and gemm(K=0) == INV
    for name in ("q", "qs", "w", "ws", "out"):
        assert gemm(**{name: 0}) == INV, name
        assert gemm(**{name: 0x1000002}) == INV, name
    assert gemm(K=2056) == UNS and gemm(K=65552) == UNS and gemm(N=65537) == UNS and gemm(M=(1 << 22) + 1) == UNS
    assert gemm(out=0x100000) == INV and gemm(out=0x300000) == INV
    assert gemm(add=0xA00010) == INV and gemm(add=0xA00000, f32=1) == INV and gemm(st=0xB00002) == INV


def test_grouped_refusals():
    lib = moe.load()

    def gg(x=0x100000, w=0x10000000, off=0x200000, ids=0x300000, y=0x400000, f32=0, sw=0, M=8, N=512, K=1024, E=16, k=4,
           st=0):
        n = lambda v: P(v) if v else None  # noqa: E731
        return lib.moe_grouped_gemm(n(x), n(w), n(off), n(ids), n(y), f32, sw, M, N, K, E, k, n(st), None)

    assert gg(M=0) == OK and gg(M=0, x=0, y=0) == OK
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(E=0), dict(k=0), dict(x=0), dict(w=0), dict(off=0), dict(y=0),
               dict(x=0x100008), dict(w=0x10000004), dict(y=0x400008), dict(off=0x200002), dict(ids=0x300001),
               dict(st=0x500002), dict(y=0x100000), dict(y=0x10000100), dict(y=0x200000), dict(y=0x300000 - 64)):
        assert gg(**kw) == INV, kw
    for kw in (dict(K=1020), dict(K=65544), dict(N=65552), dict(E=1025), dict(k=33), dict(M=1 << 21)):
        assert gg(**kw) == UNS, kw


def test_status_words_inside_the_operands_are_refused():
    # the status is cleared before the kernel reads its operands
    lib, n = moe.load(), (lambda v: P(v) if v else None)
    for st in (0x100000, 0x200004, 0x300000 + 512 * 2048 - 4, 0x900010, 0xA00000, 0xB00000):
        assert lib.moe_int8_gemm(n(0x100000), n(0x200000), n(0x300000), n(0x900000), n(0xB00000), n(0xA00000), 0, 8, 512,
                                 2048, n(st), None) == INV, hex(st)
    for st in (0x100000, 0x10000000, 0x200000 + 16 * 4, 0x300000, 0x400000 + 32 * 512 * 2 - 4):
        assert lib.moe_grouped_gemm(n(0x100000), n(0x10000000), n(0x200000), n(0x300000), n(0x400000), 0, 0, 8, 512, 1024,
                                    16, 4, n(st), None) == INV, hex(st)


def test_combine_refusals():
    lib = moe.load()

    def cb(y=0x10000000, f32=0, w=0x200000, inv=0x300000, add=0, out=0x400000, M=8, H=1024, k=4):
        n = lambda v: P(v) if v else None  # noqa: E731
        return lib.moe_combine(n(y), f32, n(w), n(inv), n(add), n(out), M, H, k, None)

    assert cb(M=0) == OK and cb(M=0, y=0) == OK
    for kw in (dict(M=-1), dict(H=0), dict(k=0), dict(y=0), dict(w=0), dict(inv=0), dict(out=0), dict(y=0x10000008),
               dict(out=0x400004), dict(add=0x500008), dict(w=0x200002), dict(inv=0x300002), dict(out=0x10000000),
               dict(add=0x400010), dict(out=0x200000 - 64)):
        assert cb(**kw) == INV, kw
    for kw in (dict(H=1020), dict(H=65544), dict(k=33), dict(M=1 << 21)):
        assert cb(**kw) == UNS, kw


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    for call in (lambda: moe.moe_block_norm(x, w_pre=x[0]), lambda: moe.moe_int8_quantize(x),
                 lambda: moe.moe_int8_gemm(x.to(torch.int8), x[:, 0].float(), x.to(torch.int8), x[:, 0].float()),
                 lambda: moe.moe_grouped_gemm(x, x[None], torch.zeros(2, dtype=torch.int32)),
                 lambda: moe.moe_combine(x, x[:, :1].float(), torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.skipif(not os.path.exists(NVCC) and shutil.which("nvcc") is None, reason="needs nvcc")
def test_ragged_plans_hold_over_a_grid_of_shapes(tmp_path):
    exe = str(tmp_path / "ragged_plan_check")
    subprocess.check_call([NVCC if os.path.exists(NVCC) else shutil.which("nvcc"), "-gencode",
                           "arch=compute_100a,code=sm_100a", "-std=c++17", "-O1", "--expt-relaxed-constexpr",
                           "-I", os.path.join(ROOT, "decode_moe_layer_b200", "csrc"),
                           "-I", os.path.join(ROOT, "include"),
                           os.path.join(ROOT, "tests", "host", "ragged_plan_check.cu"), "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr
