"""Operators as the first CUDA work of a thread: a server's worker, or autograd's thread where nothing
comes between the loss and the block."""
import threading

import pytest
import torch

from tests.test_gpu_operators import ffn_inputs, int8_layer

pytestmark = pytest.mark.gpu


def in_a_fresh_thread(call):
    got = []

    def run():
        try:
            got.append(call())
        except Exception as e:                               # noqa: BLE001 (raised below)
            got.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


@pytest.mark.parametrize("T", [1, 40, 300])
def test_first_work_of_a_thread(T):
    """Each call runs first here, so that its memory comes from torch's cache there and the operator's own
    calls are the thread's first."""
    from fp8_moe_layer_b200 import ops
    x, w13, w2, dy = ffn_inputs(T, 144, 80, torch.bfloat16, 1)
    _, h = ops.moe_gated_ffn(x, w13, w2, save_h=True)
    hid, ids, w, q13, s13, q2, s2 = int8_layer(T, 144, 4, 80, 2, 1)
    off, perm, inv = ops.moe_permute(ids, 2, None, 4, d=144, F=80)
    codes, scale = ops.moe_quant_int8(x)
    ws = ops.alloc_workspace(ops.dims(T, 144, 4, 80, 2))
    for call in (lambda: ops.moe_gated_ffn(x, w13, w2),
                 lambda: ops.moe_gated_ffn_backward(dy, x, w13, w2, h),
                 lambda: ops.moe_quant_int8(x),
                 lambda: ops.moe_matmul_int8(x, q13[0], s13[0]),
                 lambda: ops.moe_matmul_int8(codes, q13[0], s13[0], x_scale=scale),
                 lambda: ops.moe_grouped_ffn_int8(hid, q13, s13, q2, s2, off, perm, 2, ws=ws),
                 lambda: ops.moe_grouped_ffn_fp8(hid, q13.view(torch.uint8), s13, q2.view(torch.uint8), s2,
                                                 off, perm, 2, ws=ws)):
        want = call()
        del want
        want = call()
        got = in_a_fresh_thread(call)
        for a, b in zip(*((t,) if torch.is_tensor(t) else t for t in (got, want))):
            assert torch.equal(a.nan_to_num(), b.nan_to_num())
