"""include/moe_ops.h: exported symbols, exact C signatures, and what the host refuses before it
touches a device (no GPU needed)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_ops.h")
FAKE = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced by the host checks
BIG = 1 << 40

SIGNATURES = {
    "moe_quant_int8": "int (*)(int64_t, int32_t, int32_t, const void*, int8_t*, float*, void*)",
    "moe_matmul_int8_workspace_bytes": "size_t (*)(int32_t, int32_t, int32_t)",
    "moe_matmul_int8": "int (*)(int32_t, int32_t, int32_t, int32_t, const void*, const int8_t*, "
                       "const float*, const int8_t*, const float*, const float*, int32_t, void*, "
                       "void*, size_t, void*)",
    "moe_grouped_ffn_int8": "int (*)(const moe_dims*, const uint16_t*, const int8_t*, "
                            "const float*, const int8_t*, const float*, const int32_t*, "
                            "const int32_t*, float*, float*, void*, size_t, void*)",
    "moe_gated_ffn_workspace_bytes": "size_t (*)(const moe_ffn_dims*)",
    "moe_gated_ffn_backward_workspace_bytes": "size_t (*)(const moe_ffn_dims*)",
    "moe_gated_ffn": "int (*)(const moe_ffn_dims*, const uint16_t*, const uint16_t*, "
                     "const uint16_t*, uint16_t*, uint16_t*, void*, size_t, void*)",
    "moe_gated_ffn_backward": "int (*)(const moe_ffn_dims*, const uint16_t*, const uint16_t*, "
                              "const uint16_t*, const uint16_t*, const uint16_t*, uint16_t*, "
                              "uint16_t*, uint16_t*, void*, size_t, void*)",
}


@pytest.fixture(scope="module")
def ops():
    from fp8_moe_layer_b200 import build
    build.build()
    from fp8_moe_layer_b200 import ops
    return ops


def test_signatures_are_those_declared_and_exported(ops, tmp_path):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text))) == sorted(SIGNATURES)
    for name, sig in SIGNATURES.items():
        inner = sig.split("(*)(", 1)[1].rsplit(")", 1)[0]
        assert len(getattr(ops.LIB, name).argtypes) == inner.count(",") + 1, name
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "sig.c"
    src.write_text("\n".join(['#include "moe_ops.h"'] + [
        sig.replace("(*)", f"(*p{i})", 1) + f" = {name};"
        for i, (name, sig) in enumerate(SIGNATURES.items())]) + "\n")
    res = subprocess.run([gcc, "-std=c11", "-Wall", "-Werror", "-c", str(src), "-o",
                          str(tmp_path / "sig.o"), f"-I{os.path.dirname(HEADER)}"],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def test_quant_int8_refusals(ops):
    q = ops.LIB.moe_quant_int8
    bad = ops.MOE_ERR_INVALID_ARG
    assert q(0, 64, 0, None, None, None, None) == ops.MOE_OK
    assert q(-1, 64, 0, FAKE, FAKE, FAKE, None) == bad
    for K in (0, 8, 100):
        assert q(4, K, 0, FAKE, FAKE, FAKE, None) == bad
    for t in (-1, 3):
        assert q(4, 64, t, FAKE, FAKE, FAKE, None) == bad
    assert q(4, 64, 0, None, FAKE, FAKE, None) == bad
    assert q(4, 64, 0, ctypes.c_void_p((1 << 20) + 8), FAKE, FAKE, None) == bad
    assert q(4, 64, 0, FAKE, ctypes.c_void_p((1 << 20) + 4), FAKE, None) == bad
    assert q(4, 64, 0, FAKE, FAKE, ctypes.c_void_p((1 << 20) + 2), None) == bad


def test_matmul_int8_refusals(ops):
    bad, ws = ops.MOE_ERR_INVALID_ARG, ops.LIB.moe_matmul_int8_workspace_bytes

    def call(T=4, N=64, K=64, xt=0, x=FAKE, c=None, xs=None, w=FAKE, wsc=FAKE, b=None, ot=0, out=FAKE,
             wsp=FAKE, n=BIG):
        return ops.LIB.moe_matmul_int8(T, N, K, xt, x, c, xs, w, wsc, b, ot, out, wsp, n, None)

    assert call(T=0, x=None, w=None, out=None, wsp=None) == ops.MOE_OK
    odd = ctypes.c_void_p((1 << 20) + 8)
    for kw in (dict(T=-1), dict(N=0), dict(N=24), dict(K=8), dict(K=72), dict(xt=3), dict(ot=-1),
               dict(ot=3), dict(x=None), dict(x=None, c=FAKE), dict(c=FAKE), dict(xs=FAKE),
               dict(w=None), dict(wsc=None), dict(out=None), dict(x=odd), dict(w=odd), dict(wsc=odd),
               dict(b=odd), dict(out=odd), dict(x=None, c=odd, xs=FAKE)):
        assert call(**kw) == bad, kw
    assert call(K=131072) == ops.MOE_ERR_UNSUPPORTED        # an int32 sum could overflow
    assert call(n=ws(4, 64, 64) - 1) == ops.MOE_ERR_WORKSPACE
    assert call(wsp=None) == ops.MOE_ERR_WORKSPACE
    assert call(wsp=odd) == ops.MOE_ERR_WORKSPACE
    assert ws(4, 64, 72) == 0 and ws(0, 64, 64) > 0
    assert ws(4096, 64, 131056) >= 4096 * 131056            # the tokens' codes


def test_grouped_ffn_int8_refusals(ops):
    bad = ops.MOE_ERR_INVALID_ARG

    def call(dm, skip=None, ws=FAKE, n=BIG):
        p = [None if i == skip else FAKE for i in range(9)]
        p[8] = None                                          # act_scale_out may be NULL
        return ops.LIB.moe_grouped_ffn_int8(ctypes.byref(dm) if dm else None, *p, ws, n, None)

    dm = ops.dims(4, 128, 8, 256, 2)
    assert call(None) == bad and call(ops.dims(4, 100, 8, 256, 2)) == bad
    for i in range(8):
        assert call(dm, skip=i) == bad, i
    assert call(dm, n=16) == ops.MOE_ERR_WORKSPACE
    assert call(ops.dims(4, 131072, 1, 16, 1)) == ops.MOE_ERR_UNSUPPORTED
    assert call(ops.dims(0, 128, 8, 256, 2), skip=0) == ops.MOE_OK


def test_gated_ffn_refusals(ops):
    bad, L = ops.MOE_ERR_INVALID_ARG, ops.LIB
    odd = ctypes.c_void_p((1 << 20) + 8)

    def fwd(dm, x=FAKE, a=FAKE, b=FAKE, y=FAKE, h=None, ws=FAKE, n=BIG):
        return L.moe_gated_ffn(ctypes.byref(dm) if dm else None, x, a, b, y, h, ws, n, None)

    def bwd(dm, dy=FAKE, x=FAKE, a=FAKE, b=FAKE, h=FAKE, g=(FAKE, FAKE, FAKE), ws=FAKE, n=BIG):
        return L.moe_gated_ffn_backward(ctypes.byref(dm) if dm else None, dy, x, a, b, h, *g, ws, n,
                                        None)

    ok = ops.FFNDims(4, 64, 128, 0, 0)
    for dm in (None, ops.FFNDims(-1, 64, 128, 0, 0), ops.FFNDims(4, 72, 128, 0, 0),
               ops.FFNDims(4, 64, 0, 0, 0), ops.FFNDims(4, 64, 128, 2, 0),
               ops.FFNDims(4, 64, 128, 0, 2), ops.FFNDims(4, 64, 120, 1, 1)):
        assert fwd(dm) == bad and bwd(dm) == bad
        ref = ctypes.byref(dm) if dm else None
        assert L.moe_gated_ffn_workspace_bytes(ref) == 0
        assert L.moe_gated_ffn_backward_workspace_bytes(ref) == 0
    for kw in ("x", "a", "b", "y"):
        assert fwd(ok, **{kw: None}) == bad and fwd(ok, **{kw: odd}) == bad
    assert fwd(ok, h=odd) == bad
    assert fwd(ok, n=L.moe_gated_ffn_workspace_bytes(ctypes.byref(ok)) - 1) == ops.MOE_ERR_WORKSPACE
    for kw in ("dy", "x", "a", "b", "h"):
        assert bwd(ok, **{kw: None}) == bad and bwd(ok, **{kw: odd}) == bad
    for i in range(3):
        assert bwd(ok, g=tuple(odd if j == i else FAKE for j in range(3))) == bad
    need = L.moe_gated_ffn_backward_workspace_bytes(ctypes.byref(ok))
    assert bwd(ok, n=need - 1) == ops.MOE_ERR_WORKSPACE and bwd(ok, ws=None) == ops.MOE_ERR_WORKSPACE
    # what is not asked for need not be there: no W13 without dx, no x without dW13 (the workspace is
    # the next thing checked)
    assert bwd(ok, a=None, g=(None, FAKE, FAKE), n=0) == ops.MOE_ERR_WORKSPACE
    assert bwd(ok, x=None, g=(FAKE, None, FAKE), n=0) == ops.MOE_ERR_WORKSPACE
    assert fwd(ops.FFNDims(0, 64, 128, 0, 0), x=None, y=None) == ops.MOE_OK


def test_binding_refuses_cpu_tensors(ops):
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.int8)
    s = torch.ones(32)
    with pytest.raises(ValueError):
        ops.moe_quant_int8(x)
    with pytest.raises(ValueError):
        ops.moe_matmul_int8(x, w, s)
    with pytest.raises(ValueError):                          # codes without their scales
        ops.moe_matmul_int8(x.to(torch.int8), w, s)
    with pytest.raises(TypeError):
        ops.moe_quant_int8(x.double())
    f = torch.zeros(64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.moe_gated_ffn(x, f, f[:, :32].contiguous())
    with pytest.raises(TypeError):
        ops.moe_gated_ffn(x.float(), f.float(), f.float())
    with pytest.raises(ValueError):
        ops.moe_gated_ffn(x, f, f, activation="relu")


def test_int8_layer_refusals(ops):
    """What would let the router read behind its weights, or a call misread its tokens."""
    E, d, F = 3, 64, 32
    rw, rb = torch.zeros(E, d), torch.zeros(E)
    q = (torch.zeros(E, 2 * F, d, dtype=torch.int8), torch.ones(E, 2 * F),
         torch.zeros(E, d, F, dtype=torch.int8), torch.ones(E, d))
    layer = ops.MoELayerInt8(rw, rb, 2, 2, *q)
    for exc, args in [(ValueError, (rw[:, :48], rb, 2, 2, *q)), (ValueError, (rw[:2], rb, 2, 2, *q)),
                      (TypeError, (rw.double(), rb, 2, 2, *q)), (ValueError, (rw, rb[:2], 2, 2, *q)),
                      (ValueError, (rw, None, 3, 2, *q)), (ValueError, (rw, None, 0, 2, *q)),
                      (ValueError, (rw, rb, 2, 2, q[0][:, :F], *q[1:])),
                      (ValueError, (rw, rb, 2, 2, *q[:2], q[2][0], q[3]))]:
        with pytest.raises(exc):
            ops.MoELayerInt8(*args)
    x, kpt = torch.zeros(5, d, dtype=torch.bfloat16), torch.ones(5, dtype=torch.int32)
    for exc, args, kw in [(TypeError, (x.half(),), {}), (ValueError, (x[:, :48],), {}),
                          (ValueError, (x[0],), {}), (TypeError, (x, kpt.long()), {}),
                          (ValueError, (x, kpt[:4]), {}), (ValueError, (x,), {"k": 3}),
                          (ValueError, (x,), {"k": 0}),
                          (ValueError, (x,), {})]:           # the last: not on a CUDA device
        with pytest.raises(exc):
            layer(*args, **kw)
