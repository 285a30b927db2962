"""64-bit references and error bounds of the int8 and 16-bit operators (``include/moe_ops.h``).

Every function returns (value in float64, bound): |operator - value| must not exceed the bound, which
adds up, element by element, what the operator's own arithmetic may be off by:

* a rounding to a type is off by at most U[type] = finfo.eps / 2 of the value (fp16 also by half of its
  smallest subnormal, 2^-25);
* a tensor-core sum of K fp32 products by at most K 2^-23 of the sum of magnitudes (each addition may
  truncate); int8 sums are exact;
* the fast exponential and division of the activations by a relative 2^-19 (fp32 steps of 2^-21 to
  2^-23, a handful of them), the tanh form's cubic argument included.
"""
from __future__ import annotations

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
ACC = 2.0 ** -23
FAST = 2.0 ** -19


def quant_int8(x: torch.Tensor):
    """Codes (float64) and scales (float64): each is an fp32 number by definition, the correctly
    rounded quotient (a 64-bit quotient of two fp32 numbers rounds to the same fp32 number)."""
    xd = x.double()
    amax = xd.abs().amax(dim=-1, keepdim=True)
    scale = torch.where(amax == 0, torch.ones_like(amax), (amax / 127.0).float().double())
    codes = torch.round((xd / scale).float().double()).clamp(-127, 127)
    return codes, scale.squeeze(-1)


def matmul_int8(codes, scale, w, w_scale, bias, out_dtype):
    prod = (codes.double() @ w.double().t()) * scale.double()[:, None] * w_scale.double()[None, :]
    out = prod if bias is None else prod + bias.double()
    # int -> fp32, the product of the scales, its product with the sum: 3 fp32 roundings of prod
    # (a fourth is spare), the bias addition one of out; then the output's rounding
    near = 4 * U[torch.float32] * prod.abs() + U[torch.float32] * out.abs()
    return out, near + U[out_dtype] * (out.abs() + near) + TINY[out_dtype]


def activation(g, act):
    """f(g) and f'(g) in float64."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    a, b = 0.7978845608028654, 0.044715
    t = torch.tanh(a * (g + b * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * a * (1 + 3 * b * g * g)


def _mm(a, b):
    """a @ b, its magnitude sum |a| @ |b| and the accumulation's bound."""
    return a @ b, ACC * a.shape[1] * (a.abs() @ b.abs())


def gated_ffn(x, w13, w2, act):
    dt, F = x.dtype, w2.shape[1]
    u, tiny = U[dt], TINY[dt]
    x, w13, w2 = x.double(), w13.double(), w2.double()
    h, eh = _mm(x, w13.t())
    g, up, eg, eu = h[:, :F], h[:, F:], eh[:, :F], eh[:, F:]
    f, _ = activation(g, act)
    a = f * up
    # |f'| < 1.13 for both activations
    ea = (1.13 * eg + FAST * f.abs()) * (up.abs() + eu) + f.abs() * eu + FAST * a.abs()
    ea = ea + u * (a.abs() + ea) + tiny                       # the operand of the second product
    y, ey = _mm(a, w2.t())
    ey = ey * (1 + u) + ea @ w2.t().abs()
    return (y, ey + u * (y.abs() + ey) + tiny), (h, eh + u * (h.abs() + eh) + tiny)


def gated_ffn_backward(dy, x, w13, w2, h, act):
    dt, F = x.dtype, w2.shape[1]
    u, tiny = U[dt], TINY[dt]
    dy, x, w13, w2, h = (t.double() for t in (dy, x, w13, w2, h))
    g, up = h[:, :F], h[:, F:]
    f, df = activation(g, act)
    da, eda = _mm(dy, w2)
    dh = torch.cat([da * up * df, da * f], dim=1)
    # f' is a sum of terms up to 1 + |g| slope in magnitude, each good to FAST
    edf = FAST * (2 + g.abs() * (1 if act == "silu" else 4 + g * g))
    edh = torch.cat([eda * up.abs() * df.abs() + (da.abs() + eda) * up.abs() * edf,
                     eda * f.abs() + FAST * (da * f).abs()], dim=1)
    edh = edh + u * (dh.abs() + edh) + tiny
    a = f * up
    ea = 2 * FAST * a.abs()
    ea = ea + u * (a.abs() + ea) + tiny

    def out(p, q, ep, eq):
        v, ev = _mm(p, q)
        ev = ev * (1 + u) + (ep @ q.abs() if ep is not None else 0) + (p.abs() @ eq if eq is not None else 0)
        return v, ev + u * (v.abs() + ev) + tiny

    return (out(dh, w13, edh, None), out(dh.t(), x, edh.t(), None), out(dy.t(), a, None, ea))


def check(got: torch.Tensor, ref, what: str, rel: float | None = None):
    """`got` within the bound everywhere, and in the 2-norm within `rel` of the value."""
    value, bound = ref
    assert got.shape == value.shape, what
    err = (got.double() - value).abs()
    over = err - bound
    assert bool((over <= 0).all()), (what, float(err.max()), float(over.max()),
                                     int((over > 0).sum()), list(value.shape))
    if rel is not None and value.numel():
        n = float(torch.linalg.norm(value))
        assert float(torch.linalg.norm(err)) <= rel * n, (what, float(torch.linalg.norm(err)) / n)


def _block_sums(p, q):
    """sum_b |p_b q_b^T| over blocks of 128 of the contraction. A split contraction adds fp32 partial
    sums P_s, each over whole blocks, so sum_s |P_s| <= this (triangle inequality)."""
    out = torch.zeros(p.shape[0], q.shape[0], dtype=torch.float64, device=p.device)
    for k in range(0, p.shape[1], 128):
        out += (p[:, k:k + 128] @ q[:, k:k + 128].t()).abs()
    return out


def expert_int8(x, w13, s13, w2, s2w):
    """One int8 expert on tokens x [n, d] (bf16): value and bound of its output rows (fp32).

    Sums. A contraction may be split into S <= 32 parts: each exact int32 part becomes fp32 and takes
    two scales (3 roundings), and the parts are added (S - 1 roundings), so a sum is off by at most
    (S + 2) u sum_s |P_s| <= 40 u sum_b |block sums|: relative to the sum itself this grows where the
    parts cancel.
    Codes. act is off by ea (the sums of h through silu, the fast activation), its quotient v = act / s2
    by ea / s2 and by the scale's relative error ds; a code can differ by one where v lies that near to
    a half."""
    F = w2.shape[1]
    u = U[torch.float32]
    q, sx = quant_int8(x)
    sh = sx[:, None] * s13.double()[None, :]
    h = (q @ w13.double().t()) * sh
    eh = 40 * u * _block_sums(q, w13.double()) * sh
    g, up, eg, eu = h[:, :F], h[:, F:], eh[:, :F], eh[:, F:]
    f = activation(g, "silu")[0]
    a = f * up
    ef = 1.1 * eg + FAST * f.abs()                    # |silu'| < 1.1
    ea = ef * (up.abs() + eu) + f.abs() * eu + 4 * u * a.abs()
    amax = a.abs().amax(dim=1, keepdim=True)
    s2 = torch.where(amax == 0, torch.ones_like(amax), amax / 127.0)
    # the largest |act + error| lies within the largest error of any element that can be the largest
    can = (a.abs() + ea >= (a.abs() - ea).amax(dim=1, keepdim=True)).double()
    ds = (can * ea).amax(dim=1, keepdim=True) / amax.clamp_min(1e-300) + 2 * u
    v = a / s2
    aq = torch.round(v)
    margin = ea / s2 + (ds + 2 * u) * v.abs()
    near = ((v.abs() - torch.floor(v.abs()) - 0.5).abs() <= margin * (1 + 1e-3)).double()
    so = s2 * s2w.double()[None, :]
    out = (aq @ w2.double().t()) * so
    flips = (near @ w2.double().abs().t()) * so
    sums = 40 * u * (_block_sums(aq, w2.double()) * so + flips)
    return out, flips * (1 + 1e-3) + out.abs() * ds * (1 + 1e-3) + sums
