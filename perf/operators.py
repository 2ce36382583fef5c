"""Cases and plain forms of the decode-time products with 4-bit weights.

Two operators:

``fmt4``  Y[M, rows] = X[M, cols] W^T with a weight kept in one of the blockwise 4-bit
          formats (Int4, FP4 E2M1, FP4 E3M0): w = v(code) * (absmax / S), one fp32 absmax
          per 64 consecutive inputs of a row, S the largest magnitude of the format.
          X is bf16, Y is bf16 or fp32.

``moe``   a whole mixture-of-experts layer with NF4 experts for a few tokens:
            logits[t, e] = sum_d X[t, d] R[e, d]
            the top_k largest logits of a token, ties to the lower expert
            p = softmax over all experts; the weights are p of the chosen ones, divided
            by their sum where `renorm` is set
            Y[t] = sum_j weight[t, j] * D_e (silu(G_e x_t) * (U_e x_t)),  e = expert[t, j]
          G, U, D are NF4 + double-quantised tensors with the experts' rows stacked:
          gate, up [E * F, D], down [E * D, F]; w = Q[code] * c,
          c = scale8 * (scale2 / 127) + offset. Outputs: Y bf16, experts int32, weights fp32.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 64
GROUP = 256          # first-level constants per second-level constant

# magnitudes of the blockwise formats by code bits 0..2; bit 3 is the sign
MAGS = {
    "int4": [0.0, 1.0, 2.0, 3.0, 4.0, 5.0, 6.0, 7.0],
    "fp4_e2m1": [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0],
    "fp4_e3m0": [0.0] + [2.0 ** (e - 7) for e in range(1, 8)],
}


def _nf4_values():
    """The 16 normal quantiles of the format, rounded to fp32: 7 negative, zero, 8 positive, at equally
    spaced probabilities up to delta, divided by the quantile at delta."""
    from statistics import NormalDist
    inv = NormalDist().inv_cdf
    delta = 1.0 - 0.5 * (1.0 / 32.0 + 1.0 / 30.0)
    top = inv(delta)
    neg = [-inv(0.5 + (delta - 0.5) * j / 7.0) / top for j in range(7, 0, -1)]
    pos = [inv(0.5 + (delta - 0.5) * j / 8.0) / top for j in range(1, 9)]
    return neg + [0.0] + pos


NF4 = [float(torch.tensor(v, dtype=torch.float64).float()) for v in _nf4_values()]


def listed():
    return [
        # one token through a square attention projection of the 7B block: latency
        dict(name="fmt4_int4_m1_4096x4096", op="fmt4", fmt="int4", m=1, rows=4096, cols=4096, out="bf16"),
        # four sequences through the 7B block's gate projection
        dict(name="fmt4_e2m1_m4_11008x4096", op="fmt4", fmt="fp4_e2m1", m=4, rows=11008, cols=4096, out="bf16"),
        # a batch of 16 through the 7B block's down projection (long rows)
        dict(name="fmt4_e3m0_m16_4096x11008", op="fmt4", fmt="fp4_e3m0", m=16, rows=4096, cols=11008, out="bf16"),
        # one token through the 70B-like block's gate projection: the stream of the weights alone
        dict(name="fmt4_int4_m1_28672x8192", op="fmt4", fmt="int4", m=1, rows=28672, cols=8192, out="bf16"),
        # odd row count, a row of an odd number of blocks, fp32 result
        dict(name="fmt4_e2m1_m3_1001x1984", op="fmt4", fmt="fp4_e2m1", m=3, rows=1001, cols=1984, out="f32"),
        # logits of nine sequences over a vocabulary
        dict(name="fmt4_int4_m9_32000x4096", op="fmt4", fmt="int4", m=9, rows=32000, cols=4096, out="f32"),
        # many small experts, one token: latency
        dict(name="moe_t1_e64k8_2048x1024", op="moe", t=1, d=2048, f=1024, e=64, k=8, renorm=False, router="bf16"),
        # few large experts (the 7B block's feed-forward shape), one token
        dict(name="moe_t1_e8k2_4096x11008", op="moe", t=1, d=4096, f=11008, e=8, k=2, renorm=True, router="bf16"),
        # the same, four sequences: most experts have a token or two
        dict(name="moe_t4_e8k2_4096x11008", op="moe", t=4, d=4096, f=11008, e=8, k=2, renorm=True, router="bf16"),
        # odd everything, fp32 router
        dict(name="moe_t7_e13k3_1088x704", op="moe", t=7, d=1088, f=704, e=13, k=3, renorm=True, router="f32"),
        # many small experts, a batch of 16: nearly every expert is read
        dict(name="moe_t16_e64k8_2048x1024", op="moe", t=16, d=2048, f=1024, e=64, k=8, renorm=False, router="bf16"),
        # few large experts, a batch of 32: every expert, about eight tokens each
        dict(name="moe_t32_e8k2_4096x11008", op="moe", t=32, d=4096, f=11008, e=8, k=2, renorm=True, router="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        while True:
            rows, cols = _log_int(rng, 64, 32768), 64 * _log_int(rng, 4, 256)
            if 1 << 19 <= rows * cols <= 28672 * 8192:
                break
        return dict(op="fmt4", fmt=rng.choice(sorted(MAGS)), m=_log_int(rng, 1, 16), rows=rows, cols=cols,
                    out=rng.choice(["bf16", "f32"]))
    while True:
        d, f, e = 64 * _log_int(rng, 8, 64), 64 * _log_int(rng, 4, 172), _log_int(rng, 4, 128)
        if e * d * f <= 8 * 4096 * 11008:
            break
    return dict(op="moe", t=_log_int(rng, 1, 32), d=d, f=f, e=e, k=rng.randint(1, min(8, e)),
                renorm=rng.random() < 0.5, router=rng.choice(["bf16", "f32"]))


# ---------------------------------------------------------------------------- inputs
def _activations(gen, m, n):
    """Hidden states: unit variance per token with a spread of token norms and a few strong channels."""
    x = torch.randn(m, n, generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn(m, 1, generator=gen, device=DEV))
    strong = torch.randint(0, n, (max(1, n // 512),), generator=gen, device=DEV)
    x[:, strong] *= 12.0
    return x.to(torch.bfloat16)


def _nf4_parts(gen, rows, cols):
    """A stored NF4 tensor of a weight of standard deviation about 0.02: codes, int8 constants, second-level
    constants, offset."""
    n = rows * cols
    nb = -(-n // BLOCK)
    nb2 = -(-nb // GROUP)
    codes = torch.randint(0, 256, (-(-n // 2),), generator=gen, device=DEV, dtype=torch.uint8)
    scale8 = (torch.randn(nb, generator=gen, device=DEV) * 40.0).clamp_(-127.0, 127.0).round_().to(torch.int8)
    scale2 = 0.02 + 0.01 * torch.rand(nb2, generator=gen, device=DEV)
    offset = torch.full((1,), 0.05, device=DEV) + 0.005 * torch.rand(1, generator=gen, device=DEV)
    return codes, scale8, scale2, offset


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "fmt4":
        rows, cols = case["rows"], case["cols"]
        x = _activations(gen, case["m"], cols)
        codes = torch.randint(0, 256, (rows * cols // 2,), generator=gen, device=DEV, dtype=torch.uint8)
        absmax = 0.05 * torch.exp(0.25 * torch.randn(rows * cols // BLOCK, generator=gen, device=DEV))
        return dict(x=x, codes=codes, absmax=absmax)
    d, f, e = case["d"], case["f"], case["e"]
    x = _activations(gen, case["t"], d)
    router = torch.randn(e, d, generator=gen, device=DEV) / math.sqrt(d)
    if case["router"] == "bf16":
        router = router.to(torch.bfloat16)
    return dict(x=x, router=router, gate=_nf4_parts(gen, e * f, d), up=_nf4_parts(gen, e * f, d),
                down=_nf4_parts(gen, e * d, f))


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if own:
        import bit_nf4_quantized_double_b200 as q
        if case["op"] == "moe":
            d, f, e = case["d"], case["f"], case["e"]
            for name, rows, cols in (("gate", e * f, d), ("up", e * f, d), ("down", e * d, f)):
                state[name] = q.NF4Tensor(rows, cols, *state[name])
            # the scratch that such a program keeps from step to step
            state["ws"] = torch.empty(q.qlora_moe_fwd_workspace(case["t"], d, f, e, case["k"]), dtype=torch.uint8,
                                      device=DEV)
        state["q"] = q
    else:
        values = NF4 if case["op"] == "moe" else MAGS[case["fmt"]] + [-v for v in MAGS[case["fmt"]]]
        state["values"] = torch.tensor(values, device=DEV)
    return state


# ---------------------------------------------------------------------------- plain form
def _unpack(codes, values):
    """fp32 value of every code, two to a byte, the first in the high half."""
    i = codes.to(torch.int32)
    return torch.stack((values[i >> 4], values[i & 15]), dim=1).reshape(-1)


def _nf4_rows(parts, values, row0, rows, cols):
    """fp32 rows [row0, row0 + rows) of a stored NF4 tensor."""
    codes, scale8, scale2, offset = parts
    first, count = row0 * cols // BLOCK, rows * cols // BLOCK
    group = torch.arange(first, first + count, device=DEV) // GROUP
    c = scale8[first:first + count].float() * (scale2[group] / 127.0) + offset
    w = _unpack(codes[row0 * cols // 2:(row0 + rows) * cols // 2], values)
    return (w.view(count, BLOCK) * c[:, None]).view(rows, cols)


def _plain_fmt4(s):
    case = s["case"]
    rows, cols = case["rows"], case["cols"]
    w = _unpack(s["codes"], s["values"]).view(-1, BLOCK) * (s["absmax"] / MAGS[case["fmt"]][7])[:, None]
    y = s["x"].float() @ w.view(rows, cols).t()
    return y if case["out"] == "f32" else y.to(torch.bfloat16)


def _plain_moe(s):
    case = s["case"]
    t, d, f, e, k = (case[i] for i in "tdfek")
    x = s["x"].float()
    # choosing experts compares neighbouring logits: 64 bits
    logits = s["x"].double() @ s["router"].double().t()
    experts = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    p = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
    weights = (p / p.sum(dim=1, keepdim=True)).gather(1, experts)
    if case["renorm"]:
        weights = weights / weights.sum(dim=1, keepdim=True)
    weights = weights.float()
    y = torch.zeros(t, d, device=DEV)
    for i in range(e):
        g = x @ _nf4_rows(s["gate"], s["values"], i * f, f, d).t()
        u = x @ _nf4_rows(s["up"], s["values"], i * f, f, d).t()
        o = (g / (1.0 + torch.exp(-g)) * u) @ _nf4_rows(s["down"], s["values"], i * d, d, f).t()
        mine = experts == i
        y += torch.where(mine.any(dim=1, keepdim=True), (weights * mine).sum(dim=1, keepdim=True) * o, 0.0)
    return dict(y=y.to(torch.bfloat16), experts=experts.to(torch.int32), weights=weights)


def run(state):
    case = state["case"]
    if not own:
        return _plain_fmt4(state) if case["op"] == "fmt4" else _plain_moe(state)
    q = state["q"]
    if case["op"] == "fmt4":
        return q.qlora_fmt4_linear_fwd(state["x"], state["codes"], state["absmax"], case["rows"], case["fmt"],
                                       out_dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16)
    y, experts, weights = q.qlora_moe_fwd(state["x"], state["router"], state["gate"], state["up"], state["down"],
                                          case["k"], renorm=case["renorm"], ws=state["ws"])
    return dict(y=y, experts=experts, weights=weights)


# ---------------------------------------------------------------------------- work and the definition in 64 bits
def work(case):
    if case["op"] == "fmt4":
        m, rows, cols = case["m"], case["rows"], case["cols"]
        return dict(bytes=rows * cols // 2 + rows * cols // BLOCK * 4 + m * cols * 2 +
                    m * rows * (4 if case["out"] == "f32" else 2), flops=2 * m * rows * cols)
    t, d, f, e, k = (case[i] for i in "tdfek")
    # experts that at least one of t tokens chooses, for choices spread evenly
    read = e * (1.0 - (1.0 - k / e) ** t)
    weights = 3 * d * f
    stored = weights / 2 + weights / BLOCK + weights / (BLOCK * GROUP) * 4
    return dict(bytes=int(read * stored) + e * d * (2 if case["router"] == "bf16" else 4) + t * d * 4 + t * k * 8,
                flops=2 * t * k * weights + 2 * t * e * d)


def exact(case, seed):
    i = _inputs(case, seed)
    x = i["x"].double()

    def nibbles(codes):
        out = torch.empty(codes.numel() * 2, dtype=torch.int64, device=DEV)
        out[0::2] = (codes >> 4).long()
        out[1::2] = (codes & 15).long()
        return out

    if case["op"] == "fmt4":
        rows, cols, m = case["rows"], case["cols"], case["m"]
        mags = torch.tensor(MAGS[case["fmt"]], dtype=torch.float64, device=DEV)
        step = i["absmax"].double().view(rows, cols // BLOCK) / mags[7]
        y = torch.empty(m, rows, dtype=torch.float64, device=DEV)
        for r0 in range(0, rows, 4096):
            r1 = min(rows, r0 + 4096)
            n = nibbles(i["codes"][r0 * cols // 2:r1 * cols // 2])
            v = (mags[n & 7] * (1 - 2 * (n >> 3))).view(r1 - r0, cols // BLOCK, BLOCK)
            y[:, r0:r1] = x @ (v * step[r0:r1, :, None]).view(r1 - r0, cols).t()
        return y
    t, d, f, e, k = (case[j] for j in "tdfek")
    q = torch.tensor(NF4, dtype=torch.float64, device=DEV)

    def matrix(parts, expert, rows, cols):
        codes, scale8, scale2, offset = parts
        n = rows * cols
        b0, b1 = expert * n // BLOCK, (expert + 1) * n // BLOCK
        c = scale2.double().repeat_interleave(GROUP)[b0:b1] * scale8[b0:b1].double() / 127.0 + offset.double()
        return (q[nibbles(codes[expert * n // 2:(expert + 1) * n // 2])].view(-1, BLOCK) * c[:, None]).view(rows, cols)

    logits = x @ i["router"].double().t()
    prob = torch.softmax(logits, dim=1)
    experts = torch.empty(t, k, dtype=torch.int32)
    for row, values in enumerate(logits.tolist()):
        experts[row] = torch.tensor(sorted(range(e), key=lambda j: (-values[j], j))[:k], dtype=torch.int32)
    experts = experts.to(DEV)
    weights = torch.gather(prob, 1, experts.long())
    if case["renorm"]:
        weights = weights / weights.sum(dim=1, keepdim=True)
    y = torch.zeros(t, d, dtype=torch.float64, device=DEV)
    for j in sorted(set(experts.flatten().tolist())):
        tok, slot = torch.nonzero(experts == j, as_tuple=True)
        xs = x[tok]
        g = xs @ matrix(i["gate"], j, f, d).t()
        h = g * torch.sigmoid(g) * (xs @ matrix(i["up"], j, f, d).t())
        y.index_add_(0, tok, weights[tok, slot][:, None] * (h @ matrix(i["down"], j, d, f).t()))
    return dict(y=y, experts=experts, weights=weights)
