"""How the operators around the layer refuse and fail, as far as it needs no GPU."""
import ctypes
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest
import torch

import decode_moe_layer_b200 as moe

P = ctypes.c_void_p
INV, UNS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE


def test_norm_selftest_refusals():
    def call(x=0x1000000, w=0x3000000, h=0x4000000, M=592, H=512):
        n = lambda v: P(v) if v else None  # noqa: E731
        return moe.load().moe_selftest_norm_timeout(n(x), None, None, n(w), None, n(h), None, None, M, H, None)

    assert call(M=0) == INV and call(M=-1) == INV and call(H=0) == INV
    assert call(M=591) == UNS and call(M=148, H=8192) == UNS and call(H=516) == UNS
    assert call(x=0) == INV and call(w=0) == INV and call(h=0) == INV and call(h=0x1000010) == INV


def test_product_selftest_refusals():
    n = lambda v: P(v) if v else None  # noqa: E731

    def call(int8=0, x=0x1000000, off=0x5000000, y=0x4000000, st=0x6000000, M=64, N=512, K=1024, E=4):
        return moe.load().moe_selftest_product_timeout(int8, n(x), n(0x7000000), n(0x10000000), n(0x8000000), n(off), None,
                                                       n(y), 0, 0, M, N, K, E, 1, n(st), None)

    for int8 in (0, 1):
        assert call(int8, M=0) == INV and call(int8, st=0) == INV and call(int8, x=0) == INV and call(int8, y=0) == INV
        assert call(int8, st=0x4000000) == INV and call(int8, K=1020) == UNS
        assert call(int8, M=4, E=64) == UNS            # by rows: nothing is waited for
    assert call(0, off=0) == INV and call(0, M=64, E=96) == UNS


@pytest.mark.parametrize("binding", ["missing", "broken"])
def test_without_the_binding_the_layer_imports_and_the_operators_say_what_to_do(tmp_path, binding):
    here = os.path.dirname(moe.LIB_PATH)
    pkg = tmp_path / "decode_moe_layer_b200"
    pkg.mkdir()
    for f in os.listdir(here):
        if f.endswith(".py"):
            shutil.copy(os.path.join(here, f), str(pkg))
    os.symlink(moe.LIB_PATH, str(pkg / "libmoe.so"))
    if binding == "broken":
        (pkg / "_ops.so").write_bytes(b"no library")
    code = """
import torch, decode_moe_layer_b200 as moe
assert moe.__file__.startswith(%r)
assert moe.moe_workspace_bytes(2, 1024, 512, 16, 4) > 0 and callable(moe.moe_mxfp4_forward)
x = torch.zeros(2, 32)
for call in (lambda: moe.moe_block_norm(x), lambda: moe.moe_int8_quantize(x), lambda: moe.moe_int8_gemm(x, x, x, x),
             lambda: moe.moe_grouped_gemm(x, x, x), lambda: moe.moe_combine(x, x, x)):
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e) and e.__cause__ is not None, e
    else:
        raise AssertionError("no error")
print("ok")
""" % str(tmp_path)
    r = subprocess.run([sys.executable, "-c", code], cwd=str(tmp_path), capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=str(tmp_path)))
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_binding_is_rebuilt_for_another_torch_or_command(tmp_path, monkeypatch):
    path = os.path.join(os.path.dirname(moe.LIB_PATH), "build.py")
    spec = importlib.util.spec_from_file_location("_binding_build", path)
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    calls = []

    def compile_(command):
        calls.append(command)
        with open(command[command.index("-o") + 1], "w") as f:
            f.write("binding")

    src = tmp_path / "python_ops.cpp"
    src.write_text("source")
    monkeypatch.setattr(b.subprocess, "check_call", compile_)
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_ops.so"))
    monkeypatch.setattr(b, "BINDING_KEY", str(tmp_path / "objects" / "_ops.key"), raising=False)
    monkeypatch.setattr(b, "BINDING_SRC", str(src))
    for _ in range(2):
        assert b.build_binding() == b.BINDING
    assert len(calls) == 1                                    # kept
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        b.build_binding()
        b.build_binding()
    assert len(calls) == 2                                    # another torch
    b.build_binding()
    assert len(calls) == 3
    with monkeypatch.context() as m:
        m.setattr(torch, "compiled_with_cxx11_abi", lambda: not torch._C._GLIBCXX_USE_CXX11_ABI)
        b.build_binding()
    assert len(calls) == 4                                    # another ABI
    b.build_binding()
    os.utime(str(src), (4e9, 4e9))
    b.build_binding()
    assert len(calls) == 6                                    # a newer source
    b.build_binding(force=True)
    assert len(calls) == 7
