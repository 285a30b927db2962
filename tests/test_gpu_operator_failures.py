"""Failures on the device that the host cannot see, and where a user finds them.

The wait-test build of the library (include/moe_testing.h) bounds every wait inside a kernel at 2 ms and
can withhold one signal of the gate/up GEMM; nothing here faults, traps or hangs the GPU."""
import ctypes

import pytest
import torch

from tests import operator_refs as R
from tests.test_gpu_operators import gen, rnd
from tests.test_gpu_operators import int8_layer as operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from fp8_moe_layer_b200 import ops
    return ops


@pytest.fixture(scope="module")
def waittest(ops):
    from fp8_moe_layer_b200 import build
    lib = ops.load_library(build.build(lib=build.LIB_WAITTEST))
    lib.moe_test_withhold_gemm_commit.argtypes = [ctypes.c_int]
    lib.moe_test_withhold_gemm_commit.restype = None
    yield lib
    lib.moe_test_withhold_gemm_commit(0)


def int8_layer(ops, T=40, d=144, F=80, E=4):
    g = gen(T)
    layer = ops.MoELayerInt8.from_weights(
        rnd(g, E, d) * 0.05, None, 2, 2, rnd(g, E, 2 * F, d) / d ** 0.5, rnd(g, E, d, F) / F ** 0.5,
        shared=(rnd(g, 2 * F, d) / d ** 0.5, rnd(g, d, F) / F ** 0.5))
    return layer, rnd(g, T, d).to(torch.bfloat16)


@pytest.mark.parametrize("late", ["routed", "shared"])
def test_either_chain_of_the_int8_layer_reports_to_its_workspace(ops, waittest, monkeypatch, late):
    """A wait that runs out in the shared expert's launches alone, or in the routed ones alone."""
    layer, x = int8_layer(ops)
    want = layer(x)
    assert ops.device_status(layer.ws) == ops.MOE_OK
    monkeypatch.setattr(ops, "LIB", waittest)
    real, calls = ops.moe_grouped_ffn_int8, []

    def grouped(*args, **kw):
        calls.append(args[1].shape[0])
        waittest.moe_test_withhold_gemm_commit(int((len(calls) == 2) == (late == "shared")))
        try:
            return real(*args, **kw)
        finally:
            waittest.moe_test_withhold_gemm_commit(0)

    monkeypatch.setattr(ops, "moe_grouped_ffn_int8", grouped)
    layer(x)
    assert calls == [4, 1]
    assert ops.device_status(layer.ws) == ops.MOE_ERR_DEVICE_TIMEOUT
    monkeypatch.undo()
    assert torch.equal(layer(x), want)                       # the context and the layer go on
    assert ops.device_status(layer.ws) == ops.MOE_OK


def test_int8_layer_gives_its_last_workspace_back_first(ops):
    """A call takes no second workspace while the last call's is still held."""
    layer, x = int8_layer(ops, T=4000, d=1024, F=512)
    layer(x)
    held = layer.ws.numel()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    layer(x)
    assert layer.ws.numel() == held
    assert torch.cuda.max_memory_allocated() - before < held


# ------------------------------------------------------------------------------ routing data out of range
# a few rows; the down product's K split; many rows (a token's codes are copied); 256-row token tiles
ROUTED = [(9, 144, 4, 80, 2), (2, 64, 4, 8208, 2), (700, 144, 64, 80, 2), (900, 144, 3, 80, 2)]


def poisoned_workspace(ops, *sizes):
    """A workspace whose bytes read as 3.0 behind the status block: what an earlier call may have left."""
    ws = ops.alloc_workspace(ops.dims(*sizes))
    ws[256:] = 0x40
    return ws


@pytest.mark.parametrize("T,d,E,F,k", ROUTED)
@pytest.mark.parametrize("bad", ["order", "count", "negative", "token"])
def test_int8_experts_write_every_row_for_bad_routing_data(ops, T, d, E, F, k, bad):
    hid, ids, _, q13, s13, q2, s2 = operands(T, d, E, F, k, 1)
    off, perm, _ = ops.moe_permute(ids, k, None, E, d=d, F=F)
    good = ops.moe_grouped_ffn_int8(hid, q13, s13, q2, s2, off, perm, k)
    o, p = off.clone(), perm.clone()
    if bad == "order":
        o[2] = o[3] + 1
    elif bad == "count":
        o[E] = T * k + 1
    elif bad == "negative":
        o[0] = -1
    else:
        p[1], p[3] = T + 5, -1
    ws = poisoned_workspace(ops, T, d, E, F, k)
    held = torch.full((T * k, d), 3.0, device="cuda")        # where the output is likely to go
    del held
    out = ops.moe_grouped_ffn_int8(hid, q13, s13, q2, s2, o, p, k, ws=ws)
    assert ops.device_status(ws) == ops.MOE_ERR_DEVICE_CHECK
    if bad == "token":
        good[[1, 3]] = 0
        assert torch.equal(out, good)
    else:
        assert (out == 0).all()


@pytest.mark.parametrize("T,d,E,F,k", ROUTED)
def test_int8_experts_behind_the_first_ones(ops, T, d, E, F, k):
    """Offsets that start behind row 0 (the rows of experts held elsewhere): those rows are zero."""
    hid, ids, _, q13, s13, q2, s2 = operands(T, d, E, F, k, 2)
    ids = (torch.arange(T, device="cuda")[:, None] + torch.arange(k, device="cuda")).int() % E
    off, perm, _ = ops.moe_permute(ids, k, None, E, d=d, F=F)
    first = 2
    ws = poisoned_workspace(ops, T, d, E - first, F, k)
    out = ops.moe_grouped_ffn_int8(hid, *(t[first:].contiguous() for t in (q13, s13, q2, s2)),
                                   off[first:].clone(), perm, k, ws=ws)
    assert ops.device_status(ws) == ops.MOE_OK
    ends = off.tolist()
    assert 0 < ends[first] < T * k and (out[:ends[first]] == 0).all()
    for e in range(first, E):
        rows = slice(ends[e], ends[e + 1])
        if ends[e] < ends[e + 1]:
            R.check(out[rows], R.expert_int8(hid[perm[rows].long()], q13[e], s13[e], q2[e], s2[e]), e)


def test_fp8_experts_write_nothing_for_bad_offsets(ops):
    """With the down product's K split: its partial sums are not read where no product ran."""
    T, d, E, F, k = 2, 64, 4, 8208, 2
    hid, ids, _, _, s13, _, s2 = operands(T, d, E, F, k, 3)
    off, perm, _ = ops.moe_permute(ids, k, None, E, d=d, F=F)
    w13 = torch.full((E, 2 * F, d), 0x38, dtype=torch.uint8, device="cuda")      # e4m3 one
    w2 = torch.full((E, d, F), 0x38, dtype=torch.uint8, device="cuda")
    off[2] = off[3] + 1
    ws = poisoned_workspace(ops, T, d, E, F, k)
    out = ops.moe_grouped_ffn_fp8(hid, w13, s13, w2, s2, off, perm, k, ws=ws)
    assert ops.device_status(ws) == ops.MOE_ERR_DEVICE_CHECK and (out == 0).all()


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
def test_bad_offsets_of_the_largest_expert_count(ops, fmt):
    """1024 experts are as many as the tile prefix has threads: its last entry, the number of tiles, is
    one more."""
    T, d, E, F, k = 4, 16, 1024, 16, 2
    hid, ids, _, q13, s13, q2, s2 = operands(T, d, E, F, k, 4)
    off, perm, _ = ops.moe_permute(ids, k, None, E, d=d, F=F)
    off[7] = off[8] + 1
    ws = poisoned_workspace(ops, T, d, E, F, k)
    if fmt == "fp8":
        out = ops.moe_grouped_ffn_fp8(hid, q13.view(torch.uint8), s13, q2.view(torch.uint8), s2, off, perm,
                                      k, ws=ws)
    else:
        out = ops.moe_grouped_ffn_int8(hid, q13, s13, q2, s2, off, perm, k, ws=ws)
    assert ops.device_status(ws) == ops.MOE_ERR_DEVICE_CHECK and (out == 0).all()


# ------------------------------------------------------------------------------ workspaces that nobody keeps
def kept_failure(ops):
    """(what is kept on the device, what is left after asking for it)."""
    return ops.device_failure(), ops.device_failure()


def failing(lib, call):
    lib.moe_test_withhold_gemm_commit(1)
    try:
        return call()
    finally:
        lib.moe_test_withhold_gemm_commit(0)


@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("which", ["forward", "function", "backward", "int8 block", "replay"])
def test_a_failure_outlives_its_workspace(ops, waittest, monkeypatch, which, T):
    """A wait that runs out in a call whose workspace is gone when it returns."""
    from fp8_moe_layer_b200.gated_ffn import GatedFFN, gated_ffn
    torch.manual_seed(0)
    monkeypatch.setattr(ops, "LIB", waittest)
    ffn = GatedFFN(144, 80)
    x = torch.randn(T, 144, device="cuda").to(torch.bfloat16)
    served, plain = ffn.to_int8(), ffn.w13.detach()
    want = ffn(x)
    ops.device_failure()
    assert kept_failure(ops) == (ops.MOE_OK, ops.MOE_OK)
    if which == "forward":
        failing(waittest, lambda: ffn(x))
    elif which == "function":
        failing(waittest, lambda: gated_ffn(x, plain, ffn.w2.detach()))
    elif which == "backward":
        failing(waittest, lambda: want.backward(want.detach()))
    elif which == "int8 block":
        failing(waittest, lambda: served(x))
    else:
        s = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.no_grad(), torch.cuda.graph(graph, stream=s):
            failing(waittest, lambda: ffn(x))
        assert kept_failure(ops) == (ops.MOE_OK, ops.MOE_OK)
        graph.replay()
    assert kept_failure(ops) == (ops.MOE_ERR_DEVICE_TIMEOUT, ops.MOE_OK)
    with torch.no_grad():
        assert torch.equal(ffn(x), want)                     # and the calls that follow are whole
    assert kept_failure(ops) == (ops.MOE_OK, ops.MOE_OK)


def test_failures_of_every_kernel_file_are_kept(ops):
    """Caller data out of range, as found by the grouping, the preparations and the combine."""
    T, d, E, F, k = 9, 144, 4, 80, 2
    hid, ids, w, q13, s13, q2, s2 = operands(T, d, E, F, k, 1)
    off, perm, inv = ops.moe_permute(ids, k, None, E, d=d, F=F)
    out = ops.moe_grouped_ffn_int8(hid, q13, s13, q2, s2, off, perm, k)
    ops.device_failure()
    wrong_id, wrong_token, wrong_row = ids.clone(), perm.clone(), inv.clone()
    wrong_id[0, 0], wrong_token[0], wrong_row[0, 0] = E + 2, T + 2, T * k + 2
    u13, u2 = q13.view(torch.uint8), q2.view(torch.uint8)
    for call in (lambda: ops.moe_permute(wrong_id, k, None, E, d=d, F=F),
                 lambda: ops.moe_grouped_ffn_int8(hid, q13, s13, q2, s2, off, wrong_token, k),
                 lambda: ops.moe_grouped_ffn_fp8(hid, u13, s13, u2, s2, off, wrong_token, k),
                 lambda: ops.moe_combine(out, w, wrong_row),
                 lambda: ops.moe_route_topk(hid, torch.zeros(E, d, device="cuda"), None, k,
                                            torch.full((T,), k + 3, device="cuda", dtype=torch.int32), k),
                 lambda: ops.moe_ep_dispatch(hid, wrong_id, w, k, None, E, 2)):
        call()
        assert ops.device_failure(clear=False) == ops.MOE_ERR_DEVICE_CHECK
        assert kept_failure(ops) == (ops.MOE_ERR_DEVICE_CHECK, ops.MOE_OK)


def test_expert_workspaces_that_are_not_their_bytes_are_refused(ops):
    T, d, E, F, k = 9, 144, 4, 80, 2
    hid, ids, _, q13, s13, q2, s2 = operands(T, d, E, F, k, 1)
    off, perm, _ = ops.moe_permute(ids, k, None, E, d=d, F=F)
    need = ops.workspace_bytes(ops.dims(T, d, E, F, k))
    for ws in (torch.empty(1, dtype=torch.uint8, device="cuda").expand(need),
               torch.empty(need, dtype=torch.uint8), torch.empty(need, dtype=torch.int8, device="cuda")):
        with pytest.raises(ValueError):
            ops.moe_grouped_ffn_int8(hid, q13, s13, q2, s2, off, perm, k, ws=ws)
