"""Pointers that the grouped FFN's kernels would read at a misaligned address are refused on the host (no
GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def ops():
    from fp8_moe_layer_b200 import build
    build.build()
    from fp8_moe_layer_b200 import ops
    return ops


@pytest.mark.parametrize("entry", ["moe_grouped_ffn_fp8", "moe_grouped_ffn_int8"])
def test_misaligned_pointers_are_refused(ops, entry):
    dm, good = ops.dims(4, 128, 8, 256, 2), 1 << 20          # never dereferenced by the host checks

    def call(which=None, by=0):
        p = [ctypes.c_void_p(good + (by if i == which else 0)) for i in range(9)]
        return getattr(ops.LIB, entry)(ctypes.byref(dm), *p, None, 0, None)

    assert call() == ops.MOE_ERR_WORKSPACE                   # the next thing checked
    # hidden, w13, its scale, w2, its scale, offsets, tokens, output, the tokens' scales
    for which, need in enumerate((16, 16, 4, 16, 4, 4, 4, 16, 4)):
        assert call(which, need // 2) == ops.MOE_ERR_INVALID_ARG, which
        assert call(which, need) == ops.MOE_ERR_WORKSPACE, which
