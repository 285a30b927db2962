"""The int8 and 16-bit operators as programs use them: together, on streams, in graphs, through
autograd, next to memory that is not theirs, with tokens that are not finite, and refused."""
import ctypes

import pytest
import torch

from tests import operator_refs as R
from tests.test_gpu_operators import DT, ffn_inputs, gen, int8_layer, rnd, routed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from fp8_moe_layer_b200 import ops
    return ops


# ------------------------------------------------------------------------------ together
def layer_reference(ops, layer, hidden, ids, w):
    """y [T, d] in 64 bits and its bound, from the routing decision."""
    T, d = hidden.shape
    w13, s13, w2, s2 = layer.experts
    y = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    bound, mag = torch.zeros_like(y), torch.zeros_like(y)
    for e in range(layer.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            o, b = R.expert_int8(hidden[t], w13[e], s13[e], w2[e], s2[e])
            c = w[t, j].double()[:, None]
            y.index_add_(0, t, c * o)
            bound.index_add_(0, t, c * b)
            mag.index_add_(0, t, (c * o).abs())
    if layer.shared is not None:
        o, b = R.expert_int8(hidden, *(p[0] for p in layer.shared))
        y, bound, mag = y + o, bound + b, mag + o.abs()
    bound = bound + 40 * R.U[torch.float32] * mag            # the combine's fp32 sum
    return y, bound + R.U[torch.bfloat16] * (y.abs() + bound)


@pytest.mark.parametrize("T,d,E,F,k,k_max,shared,elastic", [
    (1, 256, 48, 64, 3, 3, False, False), (37, 272, 6, 144, 2, 4, True, True),
    (300, 528, 4, 336, 2, 2, True, False), (900, 256, 3, 272, 2, 2, False, False)])
def test_int8_layer(ops, T, d, E, F, k, k_max, shared, elastic):
    g = gen(T)
    w13, w2 = rnd(g, E, 2 * F, d) / d ** 0.5, rnd(g, E, d, F) / F ** 0.5
    sh = (rnd(g, 2 * F, d) / d ** 0.5, rnd(g, d, F) / F ** 0.5) if shared else None
    rw, rb = rnd(g, E, d) * 0.05, rnd(g, E) * 0.1
    layer = ops.MoELayerInt8.from_weights(rw, rb, k, k_max, w13, w2, shared=sh)
    hidden = rnd(g, T, d).to(torch.bfloat16)
    kpt = (torch.randint(1, k_max + 1, (T,), generator=g, device="cuda", dtype=torch.int32)
           if elastic else None)
    y = layer(hidden, kpt)
    assert ops.device_status(layer.ws) == ops.MOE_OK
    ids, w = ops.moe_route_topk(hidden, rw, rb, k, kpt, k_max)
    R.check(y, layer_reference(ops, layer, hidden, ids, w), "layer")
    assert torch.equal(y, layer(hidden, kpt))                # the same bits again
    assert layer(hidden[:0]).shape == (0, d)


def test_train_then_serve(ops):
    """A 16-bit block takes gradient steps, its weights are quantised, the int8 block serves it."""
    from fp8_moe_layer_b200.gated_ffn import GatedFFN
    torch.manual_seed(0)
    d, F, T = 272, 336, 200
    ffn = GatedFFN(d, F)
    x = torch.randn(T, d, device="cuda").to(torch.bfloat16)
    opt = torch.optim.SGD(ffn.parameters(), lr=0.1)
    for _ in range(2):
        opt.zero_grad()
        ffn(x).float().square().mean().backward()
        assert all(p.grad.isfinite().all() and p.grad.abs().sum() > 0 for p in ffn.parameters())
        opt.step()
    q = ffn.to_int8()
    y = q(x, dtype=torch.float32)
    R.check(y, R.expert_int8(x, *(p[0] for p in q.weights)), "int8 block")
    # the product entry point takes the same codes
    h = ops.moe_matmul_int8(x, q.weights[0][0], q.weights[1][0], out_dtype=torch.float32)
    codes, scale = R.quant_int8(x)
    R.check(h, R.matmul_int8(codes, scale, q.weights[0][0], q.weights[1][0], None, torch.float32),
            "gate/up product")
    # Near the 16-bit block: a code is off by 0.29 of a step (rms), a step is 1/127 of a row maximum of
    # about 3.5 sigma, so each of the four quantised operands adds 0.8 % at random, h's share twice
    # through the gate and the product: below 3 %, here with a factor of 3.
    with torch.no_grad():
        ref = ffn(x).float()
    assert float(torch.linalg.norm(y - ref) / torch.linalg.norm(ref)) < 0.09
    with pytest.raises(ValueError):
        GatedFFN(64, 64, activation="gelu").to_int8()


# ------------------------------------------------------------------------------ gradients
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_autograd_function(ops, act):
    from fp8_moe_layer_b200.gated_ffn import gated_ffn
    x, w13, w2, dy = ffn_inputs(70, 144, 80, torch.bfloat16, 5)
    x3 = x.view(7, 10, 144).clone().requires_grad_()
    a, b = w13.clone().requires_grad_(), w2.clone().requires_grad_()
    y = gated_ffn(x3, a, b, act)
    assert y.shape == (7, 10, 144)
    y.backward(dy.view(7, 10, 144))
    _, h = ops.moe_gated_ffn(x, w13, w2, activation=act, save_h=True)
    ref = ops.moe_gated_ffn_backward(dy, x, w13, w2, h, activation=act)
    for got, want in zip((x3.grad.view(70, 144), a.grad, b.grad), ref):
        assert torch.equal(got, want)
    # a gradient of a sum arrives expanded; frozen weights get none
    a2 = w13.clone()
    x2 = x.clone().requires_grad_()
    gated_ffn(x2, a2, w2, act).sum().backward()
    want = ops.moe_gated_ffn_backward(torch.ones_like(x), x, w13, w2, h, activation=act)[0]
    assert torch.equal(x2.grad, want) and a2.grad is None
    with torch.no_grad():
        assert torch.equal(gated_ffn(x, w13, w2, act), y.detach().view(70, 144))
    with pytest.raises(RuntimeError):                        # first-order gradients only
        z = gated_ffn(x2, a, b, act)
        (g1,) = torch.autograd.grad(z.sum(), x2, create_graph=True)
        g1.sum().backward()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_against_differences(ops, act):
    """Directional differences of the 64-bit function against the kernels' fp16 gradients. The
    difference quotient is good to e^2 and is compared through <gradient, v>: the gradient's elementwise
    bound, summed against |v|."""
    T, d, F = 33, 80, 48
    x, w13, w2, dy = ffn_inputs(T, d, F, torch.float16, 11)
    _, h = ops.moe_gated_ffn(x, w13, w2, activation=act, save_h=True)
    got = ops.moe_gated_ffn_backward(dy, x, w13, w2, h, activation=act)
    bounds = [b for _, b in R.gated_ffn_backward(dy, x, w13, w2, h, act)]
    args = [t.double() for t in (x, w13, w2)]

    def loss(x, w13, w2):
        hh = x @ w13.t()
        return float(((R.activation(hh[:, :F], act)[0] * hh[:, F:]) @ w2.t() * dy.double()).sum())

    # h was rounded to fp16 before the backward pass: that moves the gradient as well; its effect on
    # <grad, v> is the difference of the two 64-bit gradients
    exact_h = args[0] @ args[1].t()
    moved = [a - b for (a, _), (b, _) in zip(R.gated_ffn_backward(dy, x, w13, w2, h, act),
                                             R.gated_ffn_backward(dy, x, w13, w2, exact_h, act))]
    g = gen(1)
    for i in range(3):
        v = torch.randn(args[i].shape, generator=g, device="cuda", dtype=torch.float64)
        e = 1e-4
        up = loss(*[a + e * v if j == i else a for j, a in enumerate(args)])
        dn = loss(*[a - e * v if j == i else a for j, a in enumerate(args)])
        diff = (up - dn) / (2 * e)
        have = float((got[i].double() * v).sum())
        room = float((bounds[i] * v.abs()).sum()) + abs(float((moved[i] * v).sum()))
        assert abs(have - diff) <= room + 1e-5 * (1 + abs(diff)), (i, have, diff, room)


def test_gradient_at_an_odd_offset(ops):
    """A gradient that arrives as a slice behind one other element is not 16-byte aligned."""
    from fp8_moe_layer_b200.gated_ffn import gated_ffn
    x, w13, w2, dy = ffn_inputs(9, 64, 48, torch.bfloat16, 2)
    a = x.clone().requires_grad_()
    one = torch.ones(1, device="cuda", dtype=torch.bfloat16)
    both = torch.cat([one, gated_ffn(a, w13, w2).reshape(-1)])
    both.backward(torch.cat([one, dy.reshape(-1)]))
    _, h = ops.moe_gated_ffn(x, w13, w2, save_h=True)
    assert torch.equal(a.grad, ops.moe_gated_ffn_backward(dy, x, w13, w2, h)[0])


def test_int8_block_takes_the_shapes_of_the_16_bit_block(ops):
    from fp8_moe_layer_b200.gated_ffn import GatedFFN
    ffn = GatedFFN(64, 48)
    q, x = ffn.to_int8(), torch.randn(3, 4, 64, device="cuda").to(torch.bfloat16)
    flat = q(x.view(12, 64))
    for v in (x, x.transpose(0, 1), x[:, :0], x[0, 0]):
        assert q(v).shape == ffn(v).shape == v.shape
    assert torch.equal(q(x).view(12, 64), flat)
    assert torch.equal(q(x.transpose(0, 1)).transpose(0, 1).reshape(12, 64), flat)


def test_no_pre_activations_without_gradients(ops, monkeypatch):
    """The block keeps h only where a backward pass can follow."""
    from fp8_moe_layer_b200.gated_ffn import GatedFFN, gated_ffn
    kept = []
    real = ops.moe_gated_ffn
    monkeypatch.setattr(ops, "moe_gated_ffn",
                        lambda *a, save_h=False, **k: kept.append(save_h) or real(*a, save_h=save_h, **k))
    ffn, x = GatedFFN(64, 48), torch.randn(5, 64, device="cuda").to(torch.bfloat16)
    y = ffn(x)
    with torch.no_grad():
        assert torch.equal(ffn(x), y) and not ffn(x).requires_grad
    with torch.inference_mode():
        ffn(x)
    gated_ffn(x, ffn.w13.detach(), ffn.w2.detach())
    assert y.requires_grad and kept == [True, False, False, False, False]


# ------------------------------------------------------------------------------ streams and graphs
def calls(ops, seed, T=40):
    """Every operator on inputs of one seed: (callable, inputs that a graph may refill)."""
    x, w13, w2, dy = ffn_inputs(T, 144, 80, torch.bfloat16, seed)
    _, h = ops.moe_gated_ffn(x, w13, w2, save_h=True)
    hid, ids, w, q13, s13, q2, s2 = int8_layer(T, 144, 6, 80, 2, seed)
    offsets, perm, inv = ops.moe_permute(ids, 2, None, 6, d=144, F=80)
    live = dict(x=x, dy=dy, h=h, hid=hid, w=w)

    def run():
        return (ops.moe_matmul_int8(live["x"], q13[0], s13[0]),
                ops.moe_gated_ffn(live["x"], w13, w2),
                *ops.moe_gated_ffn_backward(live["dy"], live["x"], w13, w2, live["h"]),
                ops.moe_combine(ops.moe_grouped_ffn_int8(live["hid"], q13, s13, q2, s2, offsets,
                                                         perm, 2), live["w"], inv))
    return run, live


@pytest.mark.parametrize("T", [1, 40, 300])
def test_side_stream_and_repeats_give_the_same_bits(ops, T):
    run, _ = calls(ops, 1, T)
    ref = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [run() for _ in range(3)]
    s.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(ref, r))


def test_two_streams_at_once(ops):
    a, _ = calls(ops, 2, 130)
    b, _ = calls(ops, 3, 17)
    ra, rb = a(), b()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(8):
        with torch.cuda.stream(sa):
            got.append((ra, a()))
        with torch.cuda.stream(sb):
            got.append((rb, b()))
    torch.cuda.synchronize()
    for ref, r in got:
        assert all(torch.equal(x, y) for x, y in zip(ref, r))


@pytest.mark.parametrize("T", [1, 40, 200])
def test_captured_and_replayed(ops, T):
    run, live = calls(ops, 4, T)
    _, other = calls(ops, 5, T)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()                                                # one-time set-up outside the capture
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = run()
    for source in (other, {k: v.clone() for k, v in live.items()}):
        for k, v in live.items():
            v.copy_(source[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        assert all(torch.equal(a, b) for a, b in zip(got, run()))


def test_layers_and_training_step_in_a_graph(ops):
    """MoELayerInt8, the int8 block, and a forward and backward pass of the 16-bit block, captured with
    no eager graph of their leaves alive."""
    from fp8_moe_layer_b200.gated_ffn import GatedFFN
    g = gen(9)
    T, d, F, E = 24, 144, 80, 4
    layer = ops.MoELayerInt8.from_weights(
        rnd(g, E, d) * 0.05, None, 2, 2, rnd(g, E, 2 * F, d) / d ** 0.5, rnd(g, E, d, F) / F ** 0.5,
        shared=(rnd(g, 2 * F, d) / d ** 0.5, rnd(g, d, F) / F ** 0.5))
    ffn = GatedFFN(d, F)
    served = ffn.to_int8()
    x = rnd(g, T, d).to(torch.bfloat16)
    dy = rnd(g, T, d).to(torch.bfloat16)

    def run():
        for p in ffn.parameters():
            p.grad = None
        y = ffn(x)
        y.backward(dy)
        return [y.detach(), *(p.grad for p in ffn.parameters()), layer(x), served(x)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = run()
    for seed in (1, 2):
        x.copy_(rnd(gen(seed), T, d))
        dy.copy_(rnd(gen(seed + 10), T, d))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        grads = [p.grad for p in ffn.parameters()]
        assert all(torch.equal(a, b) for a, b in zip(got, run()))
        for p, was in zip(ffn.parameters(), grads):
            p.grad = was                                     # the graph's own gradient buffers


def test_captured_layer_outlives_larger_calls(ops):
    """A captured call of MoELayerInt8 replays in memory of its own after a larger call and after other
    tensors took what that one gave back."""
    g = gen(3)
    d, F, E = 144, 80, 4
    layer = ops.MoELayerInt8.from_weights(rnd(g, E, d) * 0.05, None, 2, 2, rnd(g, E, 2 * F, d) / 12,
                                          rnd(g, E, d, F) / 9)
    x, big = rnd(g, 24, d).to(torch.bfloat16), rnd(g, 900, d).to(torch.bfloat16)
    want = layer(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(x)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = layer(x)
    need = ops.workspace_bytes(ops.dims(24, d, E, F, 2))
    layer(big)
    other = [torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(64)]
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and all(bool((o == 0x5A).all()) for o in other)


def test_one_workspace_for_calls_in_sequence(ops):
    """The same caller-owned workspace through different operators and sizes."""
    ws = torch.full((1 << 24,), 0x55, dtype=torch.uint8, device="cuda")
    for T in (200, 1, 17):
        x, w13, w2, dy = ffn_inputs(T, 144, 80, torch.bfloat16, T)
        y, h = ops.moe_gated_ffn(x, w13, w2, save_h=True, ws=ws)
        assert ops.device_status(ws) == ops.MOE_OK           # cleared by the call
        g = ops.moe_gated_ffn_backward(dy, x, w13, w2, h, ws=ws)
        assert ops.device_status(ws) == ops.MOE_OK
        ws[:16] = 0x55
        w = torch.randint(-9, 9, (48, 144), device="cuda", dtype=torch.int8)
        m = ops.moe_matmul_int8(x, w, torch.ones(48, device="cuda"), ws=ws)
        assert ops.device_status(ws) == ops.MOE_OK
        assert torch.equal(y, ops.moe_gated_ffn(x, w13, w2))
        assert all(torch.equal(a, b)
                   for a, b in zip(g, ops.moe_gated_ffn_backward(dy, x, w13, w2, h)))
        assert torch.equal(m, ops.moe_matmul_int8(x, w, torch.ones(48, device="cuda")))


# ------------------------------------------------------------------------------ memory around
class Guarded:
    """A buffer with sentinels before and after it."""

    def __init__(self, shape, dtype):
        n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        self.t = self.raw[4096:4096 + n].view(dtype).view(shape)

    def intact(self):
        n = self.raw.numel() - 8192
        return bool((self.raw[:4096] == 0xA5).all() and (self.raw[4096 + n:] == 0xA5).all())


@pytest.mark.parametrize("T", [1, 15, 33, 129, 301])
def test_nothing_is_written_outside_the_outputs(ops, T):
    L, st = ops.LIB, lambda: torch.cuda.current_stream().cuda_stream
    d, F, N = 144, 80, 112
    x, w13, w2, dy = ffn_inputs(T, d, F, torch.float16, T)
    p = lambda t: t.data_ptr()                               # noqa: E731
    codes, scale = Guarded((T, d), torch.int8), Guarded((T,), torch.float32)
    assert L.moe_quant_int8(T, d, 1, p(x), p(codes.t), p(scale.t), st()) == ops.MOE_OK
    w = torch.randint(-99, 99, (N, d), device="cuda", dtype=torch.int8)
    sw = torch.rand(N, device="cuda")
    outs = [codes, scale]
    for dt, t in DT.items():
        need = L.moe_matmul_int8_workspace_bytes(T, N, d)
        ws, out = Guarded((need,), torch.uint8), Guarded((T, N), t)
        for args in ((p(x), None, None), (None, p(codes.t), p(scale.t))):
            assert L.moe_matmul_int8(T, N, d, 1, *args, p(w), p(sw), p(sw), ops.DTYPES[t], p(out.t),
                                     p(ws.t), need, st()) == ops.MOE_OK
        outs += [ws, out]
    dm = ops.FFNDims(T, d, F, 1, 0)
    ref = ctypes.byref(dm)
    need = L.moe_gated_ffn_workspace_bytes(ref)
    ws, y, h = Guarded((need,), torch.uint8), Guarded((T, d), torch.float16), Guarded((T, 2 * F), torch.float16)
    assert L.moe_gated_ffn(ref, p(x), p(w13), p(w2), p(y.t), p(h.t), p(ws.t), need, st()) == ops.MOE_OK
    outs += [ws, y, h]
    need = L.moe_gated_ffn_backward_workspace_bytes(ref)
    ws = Guarded((need,), torch.uint8)
    g = [Guarded(n, torch.float16) for n in ((T, d), (2 * F, d), (d, F))]
    assert L.moe_gated_ffn_backward(ref, p(dy), p(x), p(w13), p(w2), p(h.t), *(p(a.t) for a in g),
                                    p(ws.t), need, st()) == ops.MOE_OK
    outs += [ws, *g]
    E, k = 5, 2
    hid, ids, _, q13, s13, q2, s2 = int8_layer(T, d, E, F, k, T)
    off, perm, _ = ops.moe_permute(ids, k, None, E, d=d, F=F)
    md = ops.dims(T, d, E, F, k)
    need = ops.workspace_bytes(md)
    ws, out = Guarded((need,), torch.uint8), Guarded((T * k, d), torch.float32)
    ws.t.zero_()
    assert L.moe_grouped_ffn_int8(ctypes.byref(md), p(hid), p(q13), p(s13), p(q2), p(s2), p(off), p(perm),
                                  p(out.t), None, p(ws.t), need, st()) == ops.MOE_OK
    outs += [ws, out]
    torch.cuda.synchronize()
    assert all(o.intact() for o in outs)
    assert torch.equal(y.t, ops.moe_gated_ffn(x, w13, w2))


def test_rows_behind_the_last_routed_one_are_zero(ops):
    """Unused slots (-1) leave fewer rows than T * k: the rest of expert_out is zero, for the few-row
    and the many-row preparation."""
    for T in (6, 700):
        hid, ids, w, q13, s13, q2, s2 = int8_layer(T, 144, 4, 80, 3, T)
        ids[::2, 1:] = -1
        off, perm, inv = ops.moe_permute(ids, 3, None, 4, d=144, F=80)
        out = ops.moe_grouped_ffn_int8(hid, q13, s13, q2, s2, off, perm, 3)
        R_ = int(off[4])
        assert R_ == int((ids >= 0).sum()) < T * 3
        assert (out[R_:] == 0).all() and (out[:R_].abs().sum(dim=1) > 0).all()


def test_no_token_for_any_expert(ops):
    hid, ids, w, q13, s13, q2, s2 = int8_layer(5, 144, 4, 80, 2, 0)
    ids.fill_(-1)
    off, perm, inv = ops.moe_permute(ids, 2, None, 4, d=144, F=80)
    out = ops.moe_grouped_ffn_int8(hid, q13, s13, q2, s2, off, perm, 2)
    assert (out == 0).all()
    assert (ops.moe_combine(out, w, inv) == 0).all()


def test_bad_routing_data_is_reported(ops):
    T, E, k = 9, 4, 2
    hid, ids, _, q13, s13, q2, s2 = int8_layer(T, 144, E, 80, k, 1)
    off, perm, _ = ops.moe_permute(ids, k, None, E, d=144, F=80)
    for bad in ("token", "order", "count"):
        ws = ops.alloc_workspace(ops.dims(T, 144, E, 80, k))
        o, p = off.clone(), perm.clone()
        if bad == "token":
            p[3] = T + 5
        elif bad == "order":
            o[2] = o[3] + 1
        else:
            o[E] = T * k + 1
        out = ops.moe_grouped_ffn_int8(hid, q13, s13, q2, s2, o, p, k, ws=ws)
        assert ops.device_status(ws) == ops.MOE_ERR_DEVICE_CHECK, bad
        if bad == "token":
            assert (out[3] == 0).all()


# ------------------------------------------------------------------------------ odd contents, sizes
@pytest.mark.parametrize("T", [3, 60, 200])
def test_a_non_finite_token_stays_alone(ops, T):
    x, w13, w2, _ = ffn_inputs(T, 144, 80, torch.bfloat16, 8)
    hid, ids, w, q13, s13, q2, s2 = int8_layer(T, 144, 4, 80, 2, 8)
    bad = x.clone()
    bad[1, 5] = float("nan")
    bad[2] = float("inf")
    y, yb = ops.moe_gated_ffn(x, w13, w2), ops.moe_gated_ffn(bad, w13, w2)
    m, mb = (ops.moe_matmul_int8(t, q13[0], s13[0]) for t in (x, bad))
    rest = [0, *range(3, T)]
    for good, got in ((y, yb), (m, mb)):
        assert torch.equal(good[rest], got[rest])
        assert not got[1].isfinite().any() and not got[2].isfinite().any()
    off, perm, inv = ops.moe_permute(ids, 2, None, 4, d=144, F=80)
    o = [ops.moe_combine(ops.moe_grouped_ffn_int8(t, q13, s13, q2, s2, off, perm, 2), w, inv)
         for t in (x, bad)]
    assert torch.equal(o[0][rest], o[1][rest]) and o[1][1:3].isnan().all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [6, 140])
def test_saturated_gates(ops, act, T):
    """Pre-activations far beyond where the gate saturates: f = f' = 0 below (as at -200, where both are
    0 in fp32), f = g and f' = 1 above. Only the row's own gradients see them."""
    x, w13, w2, dy = ffn_inputs(T, 64, 48, torch.bfloat16, 4)
    x, h = x.clone(), ops.moe_gated_ffn(x, w13, w2, save_h=True)[1]
    low = h.clone()
    low[::2, :48] = -200.0
    want = ops.moe_gated_ffn_backward(dy, x, w13, w2, low, activation=act)
    for g in (-1e4, -1e12, -1e19, -3e38):
        low[::2, :48] = g
        for a, b in zip(ops.moe_gated_ffn_backward(dy, x, w13, w2, low, activation=act), want):
            assert torch.equal(a, b), g
    for g in (1e4, 1e12, 1e19, 1e30):
        high = h.clone()
        high[1, 5] = g
        got = ops.moe_gated_ffn_backward(dy, x, w13, w2, high, activation=act)
        for a, (ref, _) in zip(got, R.gated_ffn_backward(dy, x, w13, w2, high, act)):
            # dh, act and the result are rounded to half a step each: below 2^-6 of the value's norm
            assert float(torch.linalg.norm(a.double() - ref)) <= float(torch.linalg.norm(ref)) / 64, g
    # and forward: a token whose gates reach -+1e30 and saturate
    big = x.clone()
    big[0] *= 1e30
    y, gh = ops.moe_gated_ffn(big, w13, w2, activation=act, save_h=True)
    a = torch.where(gh[:, :48].double() < 0, 0.0, gh[:, :48].double()) * gh[:, 48:].double()
    assert bool((a[0].abs() > 1e30).any())
    assert torch.equal(y[1:], ops.moe_gated_ffn(x, w13, w2, activation=act)[1:])


def test_no_tokens(ops):
    dev = "cuda"
    x = torch.empty(0, 64, device=dev, dtype=torch.bfloat16)
    w13, w2 = torch.randn(64, 64, device=dev).bfloat16(), torch.randn(64, 32, device=dev).bfloat16()
    q, s = ops.moe_quant_int8(x)
    assert q.shape == (0, 64) and s.shape == (0,)
    w8 = torch.ones(32, 64, dtype=torch.int8, device=dev)
    assert ops.moe_matmul_int8(x, w8, torch.ones(32, device=dev)).shape == (0, 32)
    y, h = ops.moe_gated_ffn(x, w13, w2, save_h=True)
    assert y.shape == (0, 64) and h.shape == (0, 64)
    dx, dw13, dw2 = ops.moe_gated_ffn_backward(x, x, w13, w2, h)
    assert dx.shape == (0, 64) and (dw13 == 0).all() and (dw2 == 0).all()
    from fp8_moe_layer_b200.gated_ffn import gated_ffn
    p = w13.clone().requires_grad_()
    gated_ffn(x, p, w2).sum().backward()
    assert (p.grad == 0).all()


def test_offsets_beyond_32_bits(ops):
    """Tensors of more than 2^31 elements: codes, products and pre-activations at their far end."""
    g = gen(0)
    T, K, N = 135000, 16384, 32
    tail = rnd(g, 300, K).to(torch.bfloat16)
    x = torch.zeros(T, K, device="cuda", dtype=torch.bfloat16)
    x[-300:] = tail
    w = torch.randint(-99, 99, (N, K), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand(N, generator=g, device="cuda")
    out = ops.moe_matmul_int8(x, w, ws, out_dtype=torch.float32)
    codes, scale = R.quant_int8(tail)
    R.check(out[-300:], R.matmul_int8(codes, scale, w, ws, None, torch.float32), "far rows")
    assert (out[:-300] == 0).all()
    del x, out
    T, d, F = 70000, 16, 16400
    x, w13, w2, _ = ffn_inputs(T, d, F, torch.bfloat16, 3)
    y, h = ops.moe_gated_ffn(x, w13, w2, save_h=True)
    assert h.numel() > 1 << 31
    ry, rh = R.gated_ffn(x[-200:], w13, w2, "silu")
    R.check(h[-200:], rh, "far h")
    R.check(y[-200:], ry, "far y")


# ------------------------------------------------------------------------------ refusals
def test_refusals(ops):
    dev = "cuda"
    x = torch.zeros(4, 64, device=dev, dtype=torch.bfloat16)
    w8, s8 = torch.zeros(32, 64, device=dev, dtype=torch.int8), torch.ones(32, device=dev)
    f13, f2 = torch.zeros(64, 64, device=dev).bfloat16(), torch.zeros(64, 32, device=dev).bfloat16()
    h = torch.zeros(4, 64, device=dev).bfloat16()
    flat = torch.zeros(4 * 64 + 8, device=dev, dtype=torch.bfloat16)
    off_by_two = flat[1:1 + 4 * 64].view(4, 64)
    wide = torch.zeros(4, 128, device=dev, dtype=torch.bfloat16)[:, :64]
    small = torch.empty(256, dtype=torch.uint8, device=dev)
    V, Ty, E = ValueError, TypeError, ops.MoEError
    for exc, call in [
            (V, lambda: ops.moe_matmul_int8(off_by_two, w8, s8)),
            (V, lambda: ops.moe_matmul_int8(wide, w8, s8)),
            (V, lambda: ops.moe_matmul_int8(x, w8.t(), s8)),
            (Ty, lambda: ops.moe_matmul_int8(x, w8.float(), s8)),
            (V, lambda: ops.moe_matmul_int8(x, w8, s8[:16])),
            (V, lambda: ops.moe_matmul_int8(x, w8, s8, bias=s8.cpu())),
            (Ty, lambda: ops.moe_matmul_int8(x, w8, s8.double())),
            (Ty, lambda: ops.moe_matmul_int8(x, w8, s8, out_dtype=torch.int32)),
            (V, lambda: ops.moe_matmul_int8(x, w8, s8, x_scale=s8[:4])),
            (E, lambda: ops.moe_matmul_int8(x, w8, s8, ws=small)),
            (V, lambda: ops.moe_matmul_int8(x, w8, s8, ws=small.float())),
            (E, lambda: ops.moe_matmul_int8(x[:, :40].contiguous(), w8[:, :40].contiguous(), s8)),
            (E, lambda: ops.moe_quant_int8(x[:, :24].contiguous())),
            (V, lambda: ops.moe_quant_int8(off_by_two)),
            (V, lambda: ops.moe_gated_ffn(x, f13[:32], f2)),
            (Ty, lambda: ops.moe_gated_ffn(x, f13.half(), f2)),
            (V, lambda: ops.moe_gated_ffn(x, f13, f2.t())),
            (E, lambda: ops.moe_gated_ffn(x, f13, f2, ws=small)),
            (V, lambda: ops.moe_gated_ffn_backward(x[:3], x, f13, f2, h)),
            (V, lambda: ops.moe_gated_ffn_backward(x, x, f13, f2, h[:, :32])),
            (Ty, lambda: ops.moe_gated_ffn_backward(x.float(), x, f13, f2, h)),
            (V, lambda: ops.moe_grouped_ffn_int8(x, w8, s8, w8, s8, s8, s8, 1))]:
        with pytest.raises(exc):
            call()
    off = torch.tensor([0, 4], dtype=torch.int32, device=dev)
    perm = torch.arange(4, dtype=torch.int32, device=dev)
    q13, q2 = torch.zeros(1, 64, 64, device=dev, dtype=torch.int8), torch.zeros(1, 64, 32, device=dev, dtype=torch.int8)
    s13, s2 = torch.ones(1, 64, device=dev), torch.ones(1, 64, device=dev)
    ops.moe_grouped_ffn_int8(x, q13, s13, q2, s2, off, perm, 1)
    for exc, args in [(V, (x, q13, s13, q2, s2, off, perm[:3], 1)),
                      (Ty, (x, q13, s13, q2, s2, off, perm.long(), 1)),
                      (V, (x, q13, s13, q2, s2, off[:1], perm, 1)),
                      (Ty, (x.half(), q13, s13, q2, s2, off, perm, 1)),
                      (V, (x, q13, s13[:, :32], q2, s2, off, perm, 1)),
                      (E, (x, q13, s13, q2, s2, off, perm, 0))]:
        with pytest.raises(exc):
            ops.moe_grouped_ffn_int8(*args)
    with pytest.raises(ValueError):
        ops.MoELayerInt8(s13, None, 3, 2, q13, s13, q2, s2)
    torch.cuda.synchronize()
