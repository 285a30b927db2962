"""GPU parity of every kernel instance that a size can reach (tests/test_operator_tiles.py holds the list
to that), of the pairs of type and activation, and of contents at the ends of their range, against the
64-bit references."""
import pytest
import torch

from tests import operator_refs as R
from tests import operator_tiles as S
from tests.test_gpu_operators import DT, FFN, REL16, ffn_inputs, gen, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from fp8_moe_layer_b200 import ops
    return ops


@pytest.mark.parametrize("dtype,bias", [("bf16", False), ("fp16", True), ("fp32", True)])
@pytest.mark.parametrize("T,K,N", S.MATMUL)
def test_matmul_int8(ops, T, K, N, dtype, bias):
    g = gen(T + K + N)
    x = (rnd(g, T, K) * torch.exp(rnd(g, T, 1))).to(DT[dtype])
    w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand(N, generator=g, device="cuda") * 1e-3 + 1e-4
    b = rnd(g, N) if bias else None
    codes, scale = R.quant_int8(x)
    R.check(ops.moe_matmul_int8(x, w, ws, bias=b), R.matmul_int8(codes, scale, w, ws, b, DT[dtype]),
            (T, K, N, dtype))


def check_ffn(ops, T, d, F, dtype, act):
    x, w13, w2, dy = ffn_inputs(T, d, F, DT[dtype], T + d + F)
    rel = REL16 * R.U[DT[dtype]]
    y, h = ops.moe_gated_ffn(x, w13, w2, activation=act, save_h=True)
    ry, rh = R.gated_ffn(x, w13, w2, act)
    R.check(y, ry, "y", rel)
    R.check(h, rh, "h", rel)
    assert torch.equal(y, ops.moe_gated_ffn(x, w13, w2, activation=act))
    del ry, rh
    got = ops.moe_gated_ffn_backward(dy, x, w13, w2, h, activation=act)
    for name, a, ref in zip(("dx", "dw13", "dw2"), got, R.gated_ffn_backward(dy, x, w13, w2, h, act)):
        R.check(a, ref, name, rel)


@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("fp16", "gelu")])
@pytest.mark.parametrize("T,d,F", S.FFN)
def test_gated_ffn(ops, T, d, F, dtype, act):
    check_ffn(ops, T, d, F, dtype, act)


@pytest.mark.parametrize("dtype,act", [("bf16", "gelu"), ("fp16", "silu")])
@pytest.mark.parametrize("T,d,F", FFN)
def test_gated_ffn_other_pairs_of_type_and_activation(ops, T, d, F, dtype, act):
    check_ffn(ops, T, d, F, dtype, act)


# ------------------------------------------------------------------------------ contents
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [6, 140])
def test_gates_saturated_low_take_no_part(ops, act, T):
    """f = f' = 0 exactly: those tokens' dx is zero, and the weights' gradients are the other tokens'."""
    x, w13, w2, dy = ffn_inputs(T, 64, 48, torch.bfloat16, 4)
    h = ops.moe_gated_ffn(x, w13, w2, activation=act, save_h=True)[1]
    rest = slice(1, None, 2)
    ref = R.gated_ffn_backward(dy[rest], x[rest], w13, w2, h[rest], act)
    for g in (-200.0, -1e4, -1e19, -3e38):
        h[::2, :48] = g
        dx, dw13, dw2 = ops.moe_gated_ffn_backward(dy, x, w13, w2, h, activation=act)
        assert (dx[::2] == 0).all(), g
        for name, a, r in zip(("dx", "dw13", "dw2"), (dx[rest], dw13, dw2), ref):
            R.check(a, r, (name, g))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [6, 140])
def test_gate_saturated_high_is_the_identity(ops, act, T):
    """f = g and f' = 1 for feature 5 of token 1. At 30 both hold in fp32 already, so whatever does not
    take f itself has the same bits as there."""
    x, w13, w2, dy = ffn_inputs(T, 64, 48, torch.bfloat16, 4)
    h = ops.moe_gated_ffn(x, w13, w2, activation=act, save_h=True)[1]
    h[1, 5] = 30.0
    base = ops.moe_gated_ffn_backward(dy, x, w13, w2, h, activation=act)
    for a, r in zip(base, R.gated_ffn_backward(dy, x, w13, w2, h, act)):
        R.check(a, r, "at 30")
    others, rows, cols = (torch.arange(n, device="cuda") for n in (T, 96, 48))
    others, rows, cols = others[others != 1], rows[rows != 48 + 5], cols[cols != 5]
    for g in (1e4, 1e12, 1e30):
        h[1, 5] = g
        dx, dw13, dw2 = got = ops.moe_gated_ffn_backward(dy, x, w13, w2, h, activation=act)
        assert torch.equal(dx[others], base[0][others]), g
        assert torch.equal(dw13[rows], base[1][rows]), g     # (feature 5's gate row among them)
        assert torch.equal(dw2[:, cols], base[2][:, cols]), g
        for a, r in zip(got, R.gated_ffn_backward(dy, x, w13, w2, h, act)):
            R.check(a, r, g)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [6, 140])
def test_forward_with_saturated_gates(ops, act, T):
    """Token 0 drives half of its gates to -1e30, which take no part, and half to 1e20, which its W2 columns
    bring back to ordinary size."""
    x, w13, w2, _ = ffn_inputs(T, 64, 48, torch.bfloat16, 4)
    x[:, 0] = 0
    x[0, 0] = 1e15
    w13[:24, 0], w13[24:48, 0], w13[48:, 0] = -1e15, 1e5, 0
    w2[:, 24:] *= 1e-20
    y, h = ops.moe_gated_ffn(x, w13, w2, activation=act, save_h=True)
    ry, rh = R.gated_ffn(x, w13, w2, act)
    R.check(y, ry, "y")
    R.check(h, rh, "h")
    assert (h[0, :24] < -9e29).all() and (h[0, 24:48] > 9e19).all()
    assert float(y[0].float().abs().max()) > 0.01
    w2[:, 24:] = 0
    assert (ops.moe_gated_ffn(x, w13, w2, activation=act)[0] == 0).all()


@pytest.mark.parametrize("T", [6, 140])
def test_activations_beyond_fp16(ops, T):
    """act(g) u is an operand of the second product in the operands' type: beyond 65504 it is infinite in
    fp16, for that token alone; bf16 holds it."""
    x, w13, w2, _ = ffn_inputs(T, 64, 48, torch.float16, 4)
    x[:, 0] = 0
    w13[:, 0] = 16.0
    y = ops.moe_gated_ffn(x, w13, w2)
    x[0, 0] = 20.0                                           # gate and up near 320: a product near 1e5
    got = ops.moe_gated_ffn(x, w13, w2)
    assert not got[0].isfinite().any() and torch.equal(got[1:], y[1:])
    b = [t.to(torch.bfloat16) for t in (x, w13, w2)]
    yb = ops.moe_gated_ffn(*b)
    assert yb.isfinite().all()
    R.check(yb, R.gated_ffn(*b, "silu")[0], "bf16")


@pytest.mark.parametrize("T", [383, 400, 1000])
def test_int8_block_of_a_long_batch(ops, T):
    """From 384 tokens on the block runs on the 256-row token tiles."""
    from fp8_moe_layer_b200.gated_ffn import GatedFFN
    torch.manual_seed(T)
    q = GatedFFN(272, 336).to_int8()
    x = torch.randn(T, 272, device="cuda").to(torch.bfloat16)
    R.check(q(x, dtype=torch.float32), R.expert_int8(x, *(t[0] for t in q.weights)), T)
    assert torch.equal(q(x), q(x, dtype=torch.float32).to(torch.bfloat16))
