"""The operators beside the FP8 MoE layer, as cases to be measured: the int8 product with token and
channel scales, the routed int8 expert FFN, and the 16-bit gated FFN with its backward pass.

``run`` computes them in plain torch (``own`` false) or through ``fp8_moe_layer_b200.ops`` (``own``
true); ``exact`` gives the same outputs from the definitions in 64 bits. Layer sizes are those of
the repository's workloads (DeepSeek-V3, Qwen3-30B-A3B and Mixtral shapes) or generic.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # One token through a DeepSeek-shaped gate/up projection: a decode step, latency.
        dict(name="int8_T1", op="matmul", T=1, K=7168, N=4096, dtype="bf16", bias=False),
        # A decode batch through a Mixtral-shaped gate/up projection: the weights' bytes.
        dict(name="int8_T64", op="matmul", T=64, K=4096, N=28672, dtype="fp16", bias=False),
        # A ragged batch through an odd-sized projection with bias, all in fp32.
        dict(name="int8_ragged", op="matmul", T=1003, K=2064, N=1040, dtype="fp32", bias=True),
        # A prefill chunk through the DeepSeek-shaped projection: the tensor cores.
        dict(name="int8_T8192", op="matmul", T=8192, K=7168, N=4096, dtype="bf16", bias=False),
        # Routed int8 experts, one token of the Qwen3-shaped layer: eight experts' weights.
        dict(name="experts_T1", op="experts", T=1, d=2048, E=128, F=768, k=8),
        # The Mixtral-shaped layer at a large decode batch: every expert's weights.
        dict(name="experts_T512", op="experts", T=512, d=4096, E=8, F=14336, k=2),
        # A prefill chunk of the Qwen3-shaped layer: ragged groups of rows.
        dict(name="experts_T4096", op="experts", T=4096, d=2048, E=128, F=768, k=8),
        # One token through a Mixtral-sized dense block in 16 bits: the weights' bytes.
        dict(name="ffn_T1", op="ffn", T=1, d=4096, F=14336, dtype="bf16", act="silu", save=False),
        # A ragged batch through a small block, GELU gate.
        dict(name="ffn_ragged", op="ffn", T=333, d=2048, F=784, dtype="fp16", act="gelu",
             save=False),
        # The forward pass of a training step, DeepSeek-shaped shared expert: h is kept.
        dict(name="ffn_train", op="ffn", T=8192, d=7168, F=2048, dtype="bf16", act="silu",
             save=True),
        # The backward pass of a small fine-tuning step, ragged.
        dict(name="backward_ragged", op="backward", T=501, d=2048, F=784, dtype="fp16",
             act="gelu"),
        # The backward pass of the training step.
        dict(name="backward_train", op="backward", T=8192, d=7168, F=2048, dtype="bf16",
             act="silu"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["matmul", "experts", "ffn", "backward"])
    if op == "matmul":
        while True:
            c = dict(op=op, T=_log(rng, 1, 8192), K=_log(rng, 256, 14336, 16),
                     N=_log(rng, 256, 28672, 16), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                     bias=rng.random() < 0.5)
            if c["T"] * c["K"] * c["N"] <= 8192 * 7168 * 4096:
                return c
    if op == "experts":
        while True:
            E = rng.choice([8, 16, 64, 128, 256])
            c = dict(op=op, T=_log(rng, 1, 4096), d=_log(rng, 512, 4096, 16), E=E,
                     F=_log(rng, 192, 4096, 16), k=rng.randint(1, min(8, E)))
            if (c["T"] * c["k"] * c["d"] * c["F"] <= 512 * 2 * 4096 * 14336
                    and E * c["d"] * c["F"] <= 8 * 4096 * 14336):
                return c
    while True:
        c = dict(op=op, T=_log(rng, 1, 8192), d=_log(rng, 512, 7168, 16),
                 F=_log(rng, 256, 14336, 16), dtype=rng.choice(["bf16", "fp16"]),
                 act=rng.choice(["silu", "gelu"]))
        if op == "ffn":
            c["save"] = rng.random() < 0.5
        if c["T"] * c["d"] * c["F"] <= 8192 * 7168 * 2048 and c["d"] * c["F"] <= 4096 * 14336:
            return c


# ------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    normal = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    s = dict(case=case)
    if case["op"] == "matmul":
        T, K, N, dt = case["T"], case["K"], case["N"], DTYPES[case["dtype"]]
        # hidden states whose tokens differ in size, with a few large channels
        x = normal(T, K) * torch.exp(0.5 * normal(T, 1))
        x[:, :: max(1, K // 8)] *= 8
        s["x"] = x.to(dt)
        s["w"], s["w_scale"] = _int8_weights((N, K), normal, g)
        s["bias"] = normal(N) if case["bias"] else None
    elif case["op"] == "experts":
        T, d, E, F, k = (case[n] for n in ("T", "d", "E", "F", "k"))
        s["hidden"] = normal(T, d).to(torch.bfloat16)
        s["w13"], s["w13_scale"] = _int8_weights((E, 2 * F, d), normal, g)
        s["w2"], s["w2_scale"] = _int8_weights((E, d, F), normal, g)
        # the router's decision: some experts are taken more often than others
        logits = normal(T, E) + 0.5 * normal(1, E)
        top, ids = logits.topk(k, dim=1)
        s["topk_ids"] = ids.to(torch.int32)
        s["topk_w"] = torch.softmax(top, dim=1)
        s["most"] = int(torch.bincount(ids.reshape(-1), minlength=E).max())
    else:
        T, d, F, dt = case["T"], case["d"], case["F"], DTYPES[case["dtype"]]
        s["x"] = normal(T, d).to(dt)
        s["w13"] = (normal(2 * F, d) / math.sqrt(d)).to(dt)
        s["w2"] = (normal(d, F) / math.sqrt(F)).to(dt)
        if case["op"] == "backward":
            # what the forward pass kept, and the gradient of a mean over the tokens
            s["h"] = (s["x"].float() @ s["w13"].float().t()).to(dt)
            s["dy"] = (normal(T, d) * 0.125).to(dt)
    return s


def _int8_weights(shape, normal, g):
    """Codes of normal weights, one scale for each output channel."""
    codes = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat = codes.view(-1)
    for at in range(0, flat.numel(), 1 << 27):
        part = flat[at:at + (1 << 27)]
        part.copy_((normal(part.numel()) * 32).round_().clamp_(-127, 127))
    scale = torch.rand(shape[:-1], generator=g, device="cuda") * 4e-4 + 4e-4
    return codes, scale


# ------------------------------------------------------------------------------------- one pass
def run(state):
    return globals()["_run_" + state["case"]["op"]](state)


def _quantise(x):
    """Row codes (as fp32 values) and scales; both divisions in fp32, as the definition has them."""
    amax = x.abs().amax(dim=-1, keepdim=True)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 127), torch.ones_like(amax))
    return (x / scale).round(), scale


def _run_matmul(s):
    if own:
        from fp8_moe_layer_b200 import ops
        return ops.moe_matmul_int8(s["x"], s["w"], s["w_scale"], bias=s["bias"])
    q, scale = _quantise(s["x"].float())
    out = (q @ s["w"].float().t()) * (scale * s["w_scale"])
    if s["bias"] is not None:
        out = out + s["bias"]
    return out.to(s["x"].dtype)


def _run_experts(s):
    c = s["case"]
    T, d, E, F, k = (c[n] for n in ("T", "d", "E", "F", "k"))
    if own:
        from fp8_moe_layer_b200 import ops
        if "ws" not in s:       # the layer's workspace, kept by its user
            s["ws"] = ops.alloc_workspace(ops.dims(T, d, E, F, k))
        offsets, perm, inv = ops.moe_permute(s["topk_ids"], k, None, E, d=d, F=F, ws=s["ws"])
        out = ops.moe_grouped_ffn_int8(s["hidden"], s["w13"], s["w13_scale"], s["w2"],
                                       s["w2_scale"], offsets, perm, k, ws=s["ws"])
        return ops.moe_combine(out, s["topk_w"], inv)
    q, scale = _quantise(s["hidden"].float())
    ids = s["topk_ids"].long().reshape(-1)
    order = torch.argsort(ids, stable=True)
    first = torch.searchsorted(ids[order], torch.arange(E, device="cuda"))
    place = torch.empty_like(ids)        # a pair's row among its expert's rows
    place[order] = torch.arange(ids.numel(), device="cuda") - first[ids[order]]
    token = torch.arange(T, device="cuda").repeat_interleave(k)
    xe = torch.zeros(E, s["most"], d, device="cuda")
    se = torch.ones(E, s["most"], 1, device="cuda")
    xe[ids, place] = q[token]
    se[ids, place] = scale[token]
    h = torch.bmm(xe, s["w13"].float().transpose(1, 2)) * (se * s["w13_scale"][:, None, :])
    gate, up = h[..., :F], h[..., F:]
    aq, s2 = _quantise(gate / (1 + torch.exp(-gate)) * up)
    o = torch.bmm(aq, s["w2"].float().transpose(1, 2)) * (s2 * s["w2_scale"][:, None, :])
    y = (o[ids, place].view(T, k, d) * s["topk_w"][..., None]).sum(dim=1)
    return y.to(torch.bfloat16)


def _activation(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    a, b = math.sqrt(2 / math.pi), 0.044715       # GELU, the tanh form
    th = torch.tanh(a * (g + b * g * g * g))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * a * (1 + 3 * b * g * g)


def _run_ffn(s):
    c = s["case"]
    if own:
        from fp8_moe_layer_b200 import ops
        return ops.moe_gated_ffn(s["x"], s["w13"], s["w2"], activation=c["act"],
                                 save_h=c["save"])
    F, dt = c["F"], s["x"].dtype
    h = s["x"].float() @ s["w13"].float().t()
    y = (_activation(h[:, :F], c["act"])[0] * h[:, F:]) @ s["w2"].float().t()
    return (y.to(dt), h.to(dt)) if c["save"] else y.to(dt)


def _run_backward(s):
    c = s["case"]
    if own:
        from fp8_moe_layer_b200 import ops
        return ops.moe_gated_ffn_backward(s["dy"], s["x"], s["w13"], s["w2"], s["h"],
                                          activation=c["act"])
    F, dt = c["F"], s["x"].dtype
    h, dy = s["h"].float(), s["dy"].float()
    a, da = _activation(h[:, :F], c["act"])
    up, dact = h[:, F:], dy @ s["w2"].float()
    dh = torch.cat([dact * up * da, dact * a], dim=1)
    return ((dh @ s["w13"].float()).to(dt), (dh.t() @ s["x"].float()).to(dt),
            (dy.t() @ (a * up)).to(dt))


# ------------------------------------------------------------------------------------- its size
def work(case):
    if case["op"] == "matmul":
        T, K, N, b = case["T"], case["K"], case["N"], BYTES[case["dtype"]]
        return {"bytes": T * K * b + N * K + 4 * N * (1 + case["bias"]) + T * N * b,
                "flops": 2 * T * K * N}
    if case["op"] == "experts":
        T, d, E, F, k = (case[n] for n in ("T", "d", "E", "F", "k"))
        active = E * (1 - (1 - k / E) ** T)       # experts that some token takes, as expected
        return {"bytes": active * (3 * d * F + 4 * (2 * F + d)) + T * d * 4 + T * k * 8,
                "flops": 6 * T * k * d * F}
    T, d, F = case["T"], case["d"], case["F"]
    if case["op"] == "ffn":
        return {"bytes": 2 * (2 * T * d + 3 * d * F + (2 * T * F if case["save"] else 0)),
                "flops": 6 * T * d * F}
    return {"bytes": 2 * (3 * T * d + 6 * d * F + 2 * T * F), "flops": 12 * T * d * F}


# ------------------------------------------------------------------------------------- 64 bits
def _codes64(x):
    """Codes and scales of fp64 rows: scale and quotient are fp32 numbers by definition, so each
    is the 64-bit quotient rounded to fp32."""
    top = x.abs().max(dim=-1, keepdim=True).values
    unit = torch.tensor(127.0, dtype=torch.float64, device=x.device)
    scale = torch.where(top == 0, torch.ones_like(top), (top / unit).float().double())
    return torch.round((x / scale).float()).double(), scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matmul":
        q, scale = _codes64(s["x"].double())
        out = torch.einsum("tk,nk->tn", q, s["w"].double())
        out.mul_(scale).mul_(s["w_scale"].double()[None, :])
        return out if s["bias"] is None else out.add_(s["bias"].double())
    if case["op"] == "experts":
        return _exact_experts(case, s)
    F = case["F"]
    w13, w2, x = s["w13"].double(), s["w2"].double(), s["x"].double()
    gate = lambda g: (  # noqa: E731
        torch.nn.functional.silu(g) if case["act"] == "silu"
        else torch.nn.functional.gelu(g, approximate="tanh"))
    if case["op"] == "ffn":
        h = torch.einsum("td,fd->tf", x, w13)
        y = torch.einsum("tf,df->td", gate(h[:, :F]) * h[:, F:], w2)
        return (y, h) if case["save"] else y
    h = s["h"].double().requires_grad_()
    with torch.enable_grad():
        a = gate(h[:, :F]) * h[:, F:]
        dy = s["dy"].double()
        (dh,) = torch.autograd.grad(a, h, torch.einsum("td,df->tf", dy, w2))
    return (torch.einsum("tf,fd->td", dh, w13), torch.einsum("tf,td->fd", dh, x),
            torch.einsum("td,tf->df", dy, a.detach()))


def _exact_experts(case, s):
    """Expert by expert, as the definition reads."""
    T, d, E, F = (case[n] for n in ("T", "d", "E", "F"))
    q, scale = _codes64(s["hidden"].double())
    y = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    ids = s["topk_ids"].cpu().numpy()
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        t, j = torch.from_numpy(t).cuda(), torch.from_numpy(j).cuda()
        h = (q[t] @ s["w13"][e].double().t()) * scale[t] * s["w13_scale"][e].double()
        g = h[:, :F]
        aq, s2 = _codes64(g * torch.sigmoid(g) * h[:, F:])
        o = (aq @ s["w2"][e].double().t()) * s2 * s["w2_scale"][e].double()
        y.index_add_(0, t, o * s["topk_w"][t, j].double()[:, None])
    return y
