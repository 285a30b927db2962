"""The 64-bit references of the operators, pinned on the CPU: gradients against differences and
against autograd, the activations and the quantisation against torch's own."""
import pytest
import torch

from tests import operator_refs as R


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_and_derivative(act):
    g = torch.linspace(-12, 12, 4001, dtype=torch.float64)
    f, df = R.activation(g, act)
    ref = (torch.nn.functional.silu(g) if act == "silu"
           else torch.nn.functional.gelu(g, approximate="tanh"))
    assert torch.allclose(f, ref, rtol=1e-13, atol=1e-15)
    e = 1e-5
    diff = (R.activation(g + e, act)[0] - R.activation(g - e, act)[0]) / (2 * e)
    assert float((df - diff).abs().max()) < 1e-8
    assert float(df.abs().max()) < 1.13                       # the bounds count on it


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_ffn_gradients_against_differences(act):
    g = torch.Generator().manual_seed(0)
    T, d, F = 5, 16, 32
    x, w13, w2, dy = (torch.randn(*n, generator=g, dtype=torch.float64)
                      for n in ((T, d), (2 * F, d), (d, F), (T, d)))
    w13, w2 = w13 / d ** 0.5, w2 / F ** 0.5

    def y(x, w13, w2):
        h = x @ w13.t()
        return (R.activation(h[:, :F], act)[0] * h[:, F:]) @ w2.t()

    # the references take 16-bit tensors; here only their float64 formulas matter
    R.U[torch.float64], R.TINY[torch.float64] = 0.0, 0.0
    try:
        grads = [v for v, _ in R.gated_ffn_backward(dy, x, w13, w2, x @ w13.t(), act)]
        value = R.gated_ffn(x, w13, w2, act)[0][0]
    finally:
        del R.U[torch.float64], R.TINY[torch.float64]
    assert torch.allclose(value, y(x, w13, w2), rtol=1e-12, atol=1e-12)
    args = [x, w13, w2]
    for i, grad in enumerate(grads):
        v = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
        e = 1e-5
        up = [a + e * v if j == i else a for j, a in enumerate(args)]
        dn = [a - e * v if j == i else a for j, a in enumerate(args)]
        diff = float(((y(*up) - y(*dn)) * dy).sum() / (2 * e))
        assert abs(diff - float((grad * v).sum())) < 1e-7 * (1 + abs(diff))


def test_quantisation_rounds_half_to_even_and_scales_by_127():
    x = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 0.0] * 2])
    q, s = R.quant_int8(x)
    assert float(s[0]) == 1.0
    assert q[0, :8].tolist() == [127, 0, 2, 2, 0, -2, 126, 0]
    q, s = R.quant_int8(torch.zeros(1, 16))
    assert float(s[0]) == 1.0 and (q == 0).all()


def test_block_sums_bound_every_split():
    g = torch.Generator().manual_seed(1)
    p, q = (torch.randn(n, 700, generator=g, dtype=torch.float64) for n in (3, 4))
    total = R._block_sums(p, q)
    for cut in (128, 256, 512):
        parts = (p[:, :cut] @ q[:, :cut].t()).abs() + (p[:, cut:] @ q[:, cut:].t()).abs()
        assert (parts <= total + 1e-12).all()
