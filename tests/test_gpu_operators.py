"""GPU parity of the int8 product and the 16-bit gated FFN (forward and backward) against 64-bit
references, at sizes where tiles end inside a row, a column or the contraction."""
import pytest
import torch

from tests import operator_refs as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# In the 2-norm two roundings of random sign (an intermediate operand's and the output's) stay
# below sqrt(2) x U; the fp32 sums add less than U / 8 at these sizes.
REL16 = 1.5


@pytest.fixture(scope="module")
def ops():
    from fp8_moe_layer_b200 import ops
    return ops


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *n):
    return torch.randn(*n, generator=g, device="cuda")


# ------------------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,K", [(1, 16), (3, 48), (257, 2064), (5, 8192), (2, 8208), (7, 20000), (1500, 272), (1300, 4112), (1200, 8192), (1250, 3600),
                                    (2000, 2048)])
def test_quant_int8_bit_exact(ops, rows, K, dtype):
    g = gen(rows * K)
    x = (rnd(g, rows, K) * torch.exp(2 * rnd(g, rows, 1))).to(DT[dtype])
    x[0, :3] = torch.tensor([1.0, 0.5, -1.0]) * 4        # a quotient next to a half code
    if rows > 2:
        x[2] = 0
    codes, scale = ops.moe_quant_int8(x)
    ref, rs = R.quant_int8(x)
    assert torch.equal(codes.double(), ref)
    assert torch.equal(scale.double(), rs)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quant_int8_every_16_bit_quotient(ops, dtype):
    """Every significand of a row's maximum against every value down to 2^-9 of it (below that the
    code is 0): the codes of 16-bit rows come from a corrected reciprocal, not from a division."""
    bits = 8 if dtype == "bf16" else 11
    n = 1 << (bits - 1)
    sig = torch.arange(n, 2 * n, device="cuda").float()
    down = 0.5 ** torch.arange(0, 10, device="cuda").float()
    values = (sig[None, :] * down[:, None]).reshape(-1)                # 10 n values
    scale = 2.0 ** (3 - bits)
    for lo in range(0, n, 256):
        top = sig[lo:lo + 256, None]
        x = torch.where(values[None, :] <= top, values[None, :], top)
        x = torch.cat([top.expand(-1, 16), x, -x], dim=1)
        x = (x * scale).to(DT[dtype])
        codes, s = ops.moe_quant_int8(x.contiguous())
        ref, rs = R.quant_int8(x)
        assert torch.equal(s.double(), rs)
        assert torch.equal(codes.double(), ref)


def test_quant_int8_extreme_scales(ops):
    """Rows near the ends of the exponent range, and subnormal ones."""
    g = gen(3)
    for dt in (torch.bfloat16, torch.float32):
        e = torch.tensor([-149, -140, -133, -127, -126, -100, -70, -66, -60, 0, 90, 100, 120, 127],
                         device="cuda", dtype=torch.float64)
        x = (torch.rand(len(e), 272, generator=g, device="cuda", dtype=torch.float64) * 2 - 1)
        x = (x * 2.0 ** e[:, None]).to(dt)
        codes, scale = ops.moe_quant_int8(x)
        ref, rs = R.quant_int8(x)
        live = rs > 0                                   # a scale that underflows divides by 0
        assert torch.equal(scale.double(), rs) and live.sum() >= 12
        assert torch.equal(codes.double()[live], ref[live])


def test_quant_int8_non_finite_rows(ops):
    x = torch.ones(4, 64, device="cuda", dtype=torch.bfloat16)
    x[1, 5] = float("nan")
    x[2, 6] = float("inf")
    x[3, 7], x[3, 8] = float("-inf"), float("nan")
    codes, scale = ops.moe_quant_int8(x)
    assert scale[0] == torch.tensor(1.0) / 127 and (codes[0] == 127).all()
    assert scale[1].isnan() and scale[2].isinf() and scale[3].isnan()
    assert (codes[1:] == 0).all()
    w = torch.ones(32, 64, device="cuda", dtype=torch.int8)
    out = ops.moe_matmul_int8(x, w, torch.ones(32, device="cuda"))
    assert out[0].isfinite().all() and out[1:].isnan().all()


# ------------------------------------------------------------------------------ int8 product
MATMUL = [(1, 16, 16), (1, 4096, 1040), (2, 144, 272), (8, 48, 32), (9, 1040, 48), (16, 272, 144), (16, 4112, 272),
          (3, 528, 19504), (17, 2064, 528), (128, 512, 256), (77, 272, 19504), (100, 1040, 4912),
          (129, 528, 272), (300, 4112, 1040), (1003, 2064, 1040), (2100, 1024, 4144)]


@pytest.mark.parametrize("dtype,bias", [("bf16", False), ("fp16", True), ("fp32", True),
                                        ("fp32", False)])
@pytest.mark.parametrize("T,K,N", MATMUL)
def test_matmul_int8(ops, T, K, N, dtype, bias):
    g = gen(T + K + N)
    dt = DT[dtype]
    x = (rnd(g, T, K) * torch.exp(rnd(g, T, 1))).to(dt)
    w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand(N, generator=g, device="cuda") * 1e-3 + 1e-4
    b = rnd(g, N) if bias else None
    out = ops.moe_matmul_int8(x, w, ws, bias=b)
    codes, scale = R.quant_int8(x)
    assert out.dtype == dt
    R.check(out, R.matmul_int8(codes, scale, w, ws, b, dt), (T, K, N, dtype))


@pytest.mark.parametrize("out_dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [5, 200])
def test_matmul_int8_of_codes_extreme_values(ops, T, out_dtype):
    """Codes given by the caller, -128 among them, at the largest K whose sums cannot overflow."""
    K, N = 131056, 32
    codes = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    codes[2, ::3] = 127
    xs = torch.linspace(1e-6, 2e-6, T, device="cuda")
    ws = torch.linspace(1e-6, 2e-6, N, device="cuda") * 100
    out = ops.moe_matmul_int8(codes, w, ws, x_scale=xs, out_dtype=DT[out_dtype])
    R.check(out, R.matmul_int8(codes, xs, w, ws, None, DT[out_dtype]), out_dtype)


# ------------------------------------------------------------------------------ gated FFN
FFN = [(1, 16, 16), (1, 1040, 784), (3, 64, 48), (9, 528, 112), (16, 144, 19504), (31, 272, 144), (128, 256, 256), (129, 144, 80),
       (257, 528, 336), (500, 2048, 784), (1000, 1040, 2064), (320, 1024, 576)]


def ffn_inputs(T, d, F, dt, seed):
    g = gen(seed)
    x = rnd(g, T, d).to(dt)
    w13 = (rnd(g, 2 * F, d) * (1.5 / d ** 0.5)).to(dt)
    w2 = (rnd(g, d, F) / F ** 0.5).to(dt)
    return x, w13, w2, (rnd(g, T, d) * 0.25).to(dt)


@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("fp16", "silu"), ("bf16", "gelu"),
                                       ("fp16", "gelu")])
@pytest.mark.parametrize("T,d,F", FFN)
def test_gated_ffn(ops, T, d, F, dtype, act):
    x, w13, w2, _ = ffn_inputs(T, d, F, DT[dtype], T + d + F)
    ry, rh = R.gated_ffn(x, w13, w2, act)
    rel = REL16 * R.U[DT[dtype]]
    y = ops.moe_gated_ffn(x, w13, w2, activation=act)
    R.check(y, ry, "y", rel)
    y2, h = ops.moe_gated_ffn(x, w13, w2, activation=act, save_h=True)
    assert torch.equal(y, y2)
    R.check(h, rh, "h", rel)


@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("fp16", "gelu")])
@pytest.mark.parametrize("T,d,F", FFN)
def test_gated_ffn_backward(ops, T, d, F, dtype, act):
    x, w13, w2, dy = ffn_inputs(T, d, F, DT[dtype], T + d + F)
    _, h = ops.moe_gated_ffn(x, w13, w2, activation=act, save_h=True)
    rel = REL16 * R.U[DT[dtype]]
    got = ops.moe_gated_ffn_backward(dy, x, w13, w2, h, activation=act)
    for name, a, ref in zip(("dx", "dw13", "dw2"), got,
                            R.gated_ffn_backward(dy, x, w13, w2, h, act)):
        R.check(a, ref, name, rel)
    for need in ((True, False, False), (False, True, False), (False, False, True)):
        part = ops.moe_gated_ffn_backward(dy, x, w13, w2, h, activation=act, need=need)
        for a, b, want in zip(part, got, need):
            assert torch.equal(a, b) if want else a is None


# ------------------------------------------------------------------------------ routed int8 experts
# (T, d, E, F, k): decode tiles with a K split, ragged groups, experts without a token, prefill
# tiles of 64 to 256 rows on one CTA and on pairs
EXPERTS = [(1, 64, 8, 32, 2), (1, 2048, 128, 768, 8), (5, 528, 6, 272, 3), (64, 1024, 16, 528, 4),
           (300, 528, 4, 336, 2), (700, 272, 3, 2064, 3), (1024, 272, 8, 2064, 2), (2048, 256, 8, 208, 2),
           (1500, 528, 7, 336, 3), (2100, 144, 16, 1040, 5)]


def routed(T, E, k, g):
    top, ids = (rnd(g, T, E) + rnd(g, 1, E)).topk(k, dim=1)
    return ids.to(torch.int32), torch.softmax(top, dim=1)


def int8_layer(T, d, E, F, k, seed):
    g = gen(seed)
    codes = lambda *n: (rnd(g, *n) * 36).round().clamp(-127, 127).to(torch.int8)  # noqa: E731
    scale = lambda *n: torch.rand(*n, generator=g, device="cuda") * 1e-3 + 5e-4   # noqa: E731
    x = rnd(g, T, d).to(torch.bfloat16)
    ids, w = routed(T, E, k, g)
    return x, ids, w, codes(E, 2 * F, d), scale(E, 2 * F), codes(E, d, F), scale(E, d)


@pytest.mark.parametrize("T,d,E,F,k", EXPERTS)
def test_grouped_ffn_int8(ops, T, d, E, F, k):
    x, ids, _, w13, s13, w2, s2 = int8_layer(T, d, E, F, k, T + E)
    ws = ops.alloc_workspace(ops.dims(T, d, E, F, k))
    offsets, perm, _ = ops.moe_permute(ids, k, None, E, d=d, F=F, ws=ws)
    out, xs = ops.moe_grouped_ffn_int8(x, w13, s13, w2, s2, offsets, perm, k, ws=ws,
                                       want_act_scale=True)
    assert ops.device_status(ws) == ops.MOE_OK
    assert torch.equal(xs.double(), R.quant_int8(x)[1])
    off = offsets.tolist()
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        ref = R.expert_int8(x[perm[rows].long()], w13[e], s13[e], w2[e], s2[e])
        R.check(out[rows], ref, (e, off[e], off[e + 1]))
    assert (out[off[E]:] == 0).all()
