"""What the gated FFN modules do around the library's calls, with the calls stubbed (no GPU)."""
import pytest
import torch
from torch.autograd import forward_ad


@pytest.fixture(scope="module")
def gffn():
    from fp8_moe_layer_b200 import build
    build.build()
    from fp8_moe_layer_b200 import gated_ffn
    return gated_ffn


@pytest.fixture
def stub(gffn, monkeypatch):
    """The library's forward call as torch operations that, like it, leave no derivative behind."""
    def forward(x, w13, w2, activation="silu", save_h=False, ws=None):
        with torch.no_grad(), forward_ad._set_fwd_grad_enabled(False):
            h = x @ w13.t()
            y = (torch.nn.functional.silu(h[:, :w2.shape[1]]) * h[:, w2.shape[1]:]) @ w2.t()
        return (y, h) if save_h else y
    monkeypatch.setattr(gffn.ops, "moe_gated_ffn", forward)


def weights(d=16, F=32):
    g = torch.Generator().manual_seed(0)
    return [torch.randn(*n, generator=g) for n in ((3, d), (2 * F, d), (d, F))]


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("grad", ["frozen", "leaf", "no_grad"])
def test_forward_mode_tangents_are_refused(gffn, stub, which, grad):
    """A dual tensor requires no gradient, so nothing but its tangent says that one is wanted."""
    args = weights()
    with forward_ad.dual_level():
        dual = list(args)
        dual[which] = forward_ad.make_dual(args[which], torch.ones_like(args[which]))
        if grad == "leaf":
            dual[(which + 1) % 3] = args[(which + 1) % 3].clone().requires_grad_()
        with torch.set_grad_enabled(grad != "no_grad"), pytest.raises(NotImplementedError):
            gffn.gated_ffn(*dual)
        assert gffn.gated_ffn(*args).shape == (3, 16)        # plain tensors inside a dual level
    with pytest.raises((NotImplementedError, RuntimeError)):
        torch.func.jvp(lambda t: gffn.gated_ffn(t, *args[1:]), (args[0],), (args[0],))


def test_module_refuses_forward_mode_tangents(gffn, stub):
    ffn = gffn.GatedFFN(16, 32, dtype=torch.float32, device="cpu").requires_grad_(False)
    x = weights()[0]
    with forward_ad.dual_level(), pytest.raises(NotImplementedError):
        ffn(forward_ad.make_dual(x, x))


# ------------------------------------------------------------------------------ int8 layers
def int8_weights(E, d, F):
    return (torch.zeros(E, 2 * F, d, dtype=torch.int8), torch.ones(E, 2 * F),
            torch.zeros(E, d, F, dtype=torch.int8), torch.ones(E, d))


@pytest.fixture(params=["layer", "block"])
def int8_call(gffn, monkeypatch, request):
    """An int8 layer on the CPU, its library calls stubbed."""
    ops = gffn.ops
    monkeypatch.setattr(ops, "_elsewhere", lambda device: False)
    monkeypatch.setattr(ops, "alloc_workspace",
                        lambda *a, **k: torch.zeros(256, dtype=torch.uint8))
    monkeypatch.setattr(ops, "moe_route_topk", lambda hidden, *a, **k: (
        torch.zeros(hidden.shape[0], 2, dtype=torch.int32), torch.ones(hidden.shape[0], 2)))
    monkeypatch.setattr(ops, "moe_permute", lambda *a, **k: (None, None, None))
    monkeypatch.setattr(ops, "moe_grouped_ffn_int8",
                        lambda hidden, *a, **k: torch.ones(hidden.shape))
    monkeypatch.setattr(ops, "moe_combine", lambda out, *a, **k: out.bfloat16())
    q = int8_weights(3, 64, 32)
    if request.param == "layer":
        return ops.MoELayerInt8(torch.zeros(3, 64), None, 2, 2, *q)
    return gffn.Int8GatedFFN(*(t[0] for t in q))


def test_int8_layers_refuse_inputs_whose_derivative_is_wanted(int8_call):
    """They return a tensor without a graph: the layers below would get no gradient, without a word."""
    x = torch.ones(5, 64, dtype=torch.bfloat16)
    leaf = x.clone().requires_grad_()
    for t in (leaf, leaf * 2):
        with pytest.raises(RuntimeError):
            int8_call(t)
        with torch.no_grad():
            assert int8_call(t).shape == (5, 64)
        assert int8_call(t.detach()).shape == (5, 64)
    with torch.inference_mode():
        assert int8_call(leaf).shape == (5, 64)
    with forward_ad.dual_level(), torch.no_grad(), pytest.raises(NotImplementedError):
        int8_call(forward_ad.make_dual(x, x))


def test_int8_block_is_a_module(gffn):
    """It takes the 16-bit block's place in a model, moves with it, and saves and loads with it."""
    class Layer(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.ffn = gffn.GatedFFN(64, 32, device="cpu")

    q = [t[0] for t in int8_weights(1, 64, 32)]
    q[0][3], q[1][5] = 7, 0.25
    layer = Layer()
    layer.ffn = gffn.Int8GatedFFN(*q)
    assert not list(layer.parameters())
    state = layer.state_dict()
    assert sorted(state) == ["ffn.w13", "ffn.w13_scale", "ffn.w2", "ffn.w2_scale"]
    other = Layer()
    other.ffn = gffn.Int8GatedFFN(*(t[0] for t in int8_weights(1, 64, 32)))
    other.load_state_dict(state)
    for moved in (other, other.to(torch.bfloat16), other.half(), other.double(), other.to("cpu").float()):
        for t, want in zip(moved.ffn.weights, q):
            assert t.dtype == want.dtype and torch.equal(t[0], want)
    meta = other.to("meta")
    assert all(t.device.type == "meta" for t in meta.ffn.weights)
    assert [t.dtype for t in meta.ffn.weights] == [t.dtype for t in q]


def test_workspaces_that_are_not_their_bytes_are_refused(gffn):
    """An expanded tensor has as many elements as asked for and a single byte behind them; a workspace of
    another device is not the kernels' to write."""
    ops, cpu = gffn.ops, torch.device("cpu")
    plain = torch.empty(4096, dtype=torch.uint8)
    assert ops._workspace(plain, 4096, "", cpu) is plain
    for ws in (torch.empty(1, dtype=torch.uint8).expand(4096), plain[::2], plain.view(torch.int32),
               torch.empty(4096, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError):
            ops._workspace(ws, 4096, "", cpu)
