"""Cases that measure the operators around an MoE layer's experts: the top-k gate
(with its gradient), the root-mean-square norm with the residual's addition (with
its gradient, and with 8-bit output), and a whole MoE layer for a few tokens --
router, gate, experts over 8-bit weights, weighted sum.

`run` computes either the plain form of an operator (elementary torch operations in
32 bits, in 64 where values lie next to a border, rounded once at the end) or, where
`own` is true, the calls a user makes of the library.
"""
import math

import torch

own = False

#: A block whose largest magnitude is below this is quantised as if that were its
#: largest magnitude, so that its scale stays a normal number.
AMAX_FLOOR = 2.0 ** -100
E4M3_MAX = 448.0
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one user's next token through the whole layer: the selected experts' bytes
        dict(name="layer one token", op="layer", T=1, topk=8, E=128, D=6144, I=2048, type="bf16",
             score="softmax", bias=False, renormalize=True),
        # eight users' next tokens: most routes reach an expert of their own
        dict(name="layer 8 tokens", op="layer", T=8, topk=8, E=128, D=6144, I=2048, type="bf16",
             score="sigmoid", bias=True, renormalize=True),
        # a small model with ragged widths (no multiple of 128), several tokens an expert
        dict(name="layer small ragged", op="layer", T=5, topk=2, E=8, D=1040, I=528, type="fp16",
             score="softmax", bias=False, renormalize=False),
        # one token's gate: latency
        dict(name="gate one token", op="gate", T=1, topk=8, E=128, type="fp32", score="softmax",
             bias=False, renormalize=True),
        # a prefill's gate, scores of their own and a bias that balances the experts' load
        dict(name="gate 8192", op="gate", T=8192, topk=8, E=128, type="fp32", score="sigmoid",
             bias=True, renormalize=True),
        # training of the router: an odd number of tokens and of experts
        dict(name="gate grad odd", op="gate_grad", T=1021, topk=6, E=60, type="bf16",
             score="softmax", bias=False, renormalize=False),
        # training of the router: a full batch over many experts
        dict(name="gate grad 8192", op="gate_grad", T=8192, topk=8, E=256, type="fp32",
             score="softmax", bias=False, renormalize=True),
        # one token between two layers, 8-bit output for the next projection: latency
        dict(name="norm 8-bit one token", op="norm_fp8", T=1, D=6144, type="bf16", residual=True),
        # a prefill between two layers, 8-bit output for the next projection
        dict(name="norm 8-bit 8192", op="norm_fp8", T=8192, D=6144, type="bf16", residual=True),
        # rows of an odd width in 16-bit floats, no residual
        dict(name="norm odd", op="norm", T=1021, D=2047, type="fp16", residual=False),
        # the forward pass of training, and a prefill whose next step wants plain rows
        dict(name="norm 8192", op="norm", T=8192, D=6144, type="bf16", residual=True),
        # training: gradients of the rows and of the weight
        dict(name="norm grad 8192", op="norm_grad", T=8192, D=6144, type="bf16", residual=True),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["layer", "layer", "gate", "gate_grad", "norm", "norm_grad", "norm_fp8"])
    if op == "layer":
        E = rng.choice([8, 16, 60, 64, 96, 128])
        return dict(op=op, T=rng.randint(1, 8), topk=rng.randint(1, 8), E=E,
                    D=16 * _log_uniform(rng, 8, 384), I=16 * _log_uniform(rng, 8, 128),
                    type=rng.choice(["bf16", "bf16", "fp16"]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.4,
                    renormalize=rng.random() < 0.6)
    T = _log_uniform(rng, 1, 8192)
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("gate", "gate_grad"):
        E = rng.choice([8, 16, 60, 64, 96, 128, 256])
        return dict(op=op, T=T, topk=rng.randint(1, 8), E=E, type=rng.choice(["fp32", kind]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.4,
                    renormalize=rng.random() < 0.6)
    D = _log_uniform(rng, 64, 6144)
    if op == "norm_fp8":
        return dict(op=op, T=T, D=max(64, D // 16 * 16), type=rng.choice(["bf16", "bf16", "fp16"]),
                    residual=rng.random() < 0.7)
    if rng.random() < 0.7:
        D = max(64, D // 8 * 8)
    return dict(op=op, T=T, D=D, type=kind, residual=rng.random() < 0.7)


# ------------------------------------------------------------------- inputs

def _normal(gen, shape, kind, sigma=1.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x.mul_(sigma) if sigma != 1.0 else x).to(TYPES[kind])


def _weights(gen, E, N, K):
    """E4M3 weights ~ N(0, 0.02) [E, N, K] and their scales, one for each
    block of 128 x 128."""
    nb, kb = -(-N // 128), -(-K // 128)
    codes = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((E, nb, kb), dtype=torch.float32, device="cuda")
    for e in range(E):
        w = torch.zeros((nb * 128, kb * 128), dtype=torch.float32, device="cuda")
        w[:N, :K] = torch.randn((N, K), generator=gen, device="cuda").mul_(0.02)
        blocks = w.view(nb, 128, kb, 128)
        amax = blocks.abs().amax(dim=(1, 3))
        scales[e] = amax / E4M3_MAX
        q = (blocks / scales[e][:, None, :, None]).clamp_(-E4M3_MAX, E4M3_MAX)
        codes[e] = q.view(nb * 128, kb * 128)[:N, :K].to(torch.float8_e4m3fn)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, kind, T = case["op"], case["type"], case["T"]
    s = {"op": op}
    if op in ("layer", "gate", "gate_grad"):
        E = case["E"]
        s.update(topk=case["topk"], score=case["score"], renormalize=case["renormalize"],
                 scale=2.5 if case["score"] == "sigmoid" else 1.0)
        # as large as the differences between the scores: it changes which experts win
        s["bias"] = (torch.randn(E, generator=gen, device="cuda").mul_(0.05) if case["bias"]
                     else None)
        if op == "layer":
            D = case["D"]
            s["x"] = _normal(gen, (T, D), kind)
            s["router"] = _normal(gen, (E, D), kind, D ** -0.5)
            s["gate_up"] = _weights(gen, E, 2 * case["I"], D)
            s["down"] = _weights(gen, E, D, case["I"])
            return s
        s["logits"] = _normal(gen, (T, E), kind, 1.5)
        if op == "gate_grad":
            s["ids"] = _plain_gate(s["logits"], s)[0]
            s["dweights"] = _normal(gen, (T, case["topk"]), "fp32")
        return s
    D = case["D"]
    s["weight"] = (1.0 + _normal(gen, (D,), "fp32", 0.1)).to(TYPES[kind])
    s["residual"] = _normal(gen, (T, D), kind, 2.0) if case["residual"] else None
    if op == "norm_grad":
        s["h"] = _normal(gen, (T, D), kind, 2.0)
        s["dy"] = _normal(gen, (T, D), kind)
        # the gradient that reaches the sum by the residual's own way
        s["dh"] = s.pop("residual")
    else:
        s["x"] = _normal(gen, (T, D), kind)
    return s


# --------------------------------------------------------------- plain forms

def _plain_scores(logits, score):
    l = logits.double()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    p = torch.exp(l - l.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def _plain_gate(logits, s):
    """The experts (best first, the lower number first among equals) and weights."""
    scores = _plain_scores(logits, s["score"])
    key = logits.double() if s["bias"] is None else scores + s["bias"].double()
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :s["topk"]]
    w = scores.gather(1, ids)
    if s["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), (w * s["scale"]).float()


def _plain_gate_grad(s):
    logits, ids = s["logits"], s["ids"].long()
    p = _plain_scores(logits, s["score"])
    w = p.gather(1, ids)
    g = s["dweights"].double() * s["scale"]
    if s["renormalize"]:
        total = w.sum(1, keepdim=True)
        g = (g - (g * w).sum(1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter(1, ids, g)
    if s["score"] == "sigmoid":
        dl = dp * p * (1.0 - p)
    else:
        dl = p * (dp - (dp * p).sum(1, keepdim=True))
    return dl.to(logits.dtype)


def _plain_sum(s):
    return s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)


def _plain_unrounded(h, weight):
    h = h.float()
    return h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * weight.float()


def _plain_blocks(x):
    """E4M3 codes (as values, 32 bits) and 1 x 128 scales [blocks, rows] of rows x."""
    M, K = x.shape
    kb = -(-K // 128)
    blocks = torch.nn.functional.pad(x.float(), (0, kb * 128 - K)).view(M, kb, 128)
    amax = blocks.abs().amax(2, keepdim=True).clamp(min=AMAX_FLOOR)
    q = (blocks * E4M3_MAX / amax).to(torch.float8_e4m3fn)
    return q.view(M, kb * 128)[:, :K], (amax / E4M3_MAX)[:, :, 0]


def _plain_quantise(x):
    """x as the values that its E4M3 codes and 1 x 128 scales stand for."""
    q, scale = _plain_blocks(x)
    return q.float() * scale.repeat_interleave(128, 1)[:, :x.shape[1]]


def _plain_norm(s):
    h = _plain_sum(s)
    y = _plain_unrounded(h, s["weight"]).to(h.dtype)
    return y if s["residual"] is None else (y, h)


def _plain_norm_fp8(s):
    h = _plain_sum(s)
    q, scale = _plain_blocks(_plain_unrounded(h, s["weight"]))
    q, scale = q.contiguous(), scale.t().contiguous()
    return (q, scale) if s["residual"] is None else (q, scale, h)


def _plain_norm_grad(s):
    h, dy, weight = s["h"].float(), s["dy"].float(), s["weight"].float()
    rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    g = dy * weight
    dx = rstd * (g - h * (rstd * rstd * (g * h).mean(1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    dw = (dy * h * rstd).double().sum(0)
    return dx.to(s["h"].dtype), dw.to(s["weight"].dtype)


def _plain_routes_weights(pair, ids):
    """Each route's weights in 32 bits [R, N, K]."""
    codes, scales = pair
    N, K = codes.shape[1:]
    wide = scales[ids].repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    return codes.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * wide


def _plain_layer(s):
    x = s["x"]
    T, topk = x.shape[0], s["topk"]
    logits = x.double() @ s["router"].double().t()
    ids, weights = _plain_gate(logits, s)
    ids = ids.long().reshape(-1)
    rows = _plain_quantise(x).repeat_interleave(topk, 0)
    gate, up = torch.bmm(_plain_routes_weights(s["gate_up"], ids), rows[:, :, None])[:, :, 0].chunk(2, 1)
    h = _plain_quantise(gate / (1.0 + torch.exp(-gate)) * up)
    y = torch.bmm(_plain_routes_weights(s["down"], ids), h[:, :, None])[:, :, 0]
    return (y.view(T, topk, -1) * weights[:, :, None]).sum(1).to(x.dtype)


def _run_plain(s):
    op = s["op"]
    if op == "layer":
        return _plain_layer(s)
    if op == "gate":
        return _plain_gate(s["logits"], s)
    if op == "gate_grad":
        return _plain_gate_grad(s)
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_fp8":
        return _plain_norm_fp8(s)
    return _plain_norm_grad(s)


def _run_own(s):
    from moe_grouped_gemm_nvfp4_gb300 import gating, moe, norm
    op = s["op"]
    if op in ("layer", "gate", "gate_grad"):
        how = dict(bias=s["bias"], score=s["score"], renormalize=s["renormalize"], scale=s["scale"])
        if op == "layer":
            return moe.Fp8MoE(s["router"], s["gate_up"], s["down"], s["topk"], **how).step(s["x"])
        if op == "gate":
            return gating.topk_gate(s["logits"], s["topk"], **how)
        del how["bias"]                      # it chooses the experts; the weights do not hold it
        return gating.topk_gate_grad(s["dweights"], s["logits"], s["ids"], **how)
    if op == "norm":
        return norm.rms_norm(s["x"], s["weight"], s["residual"], eps=EPS)
    if op == "norm_fp8":
        return norm.rms_norm_fp8(s["x"], s["weight"], s["residual"], eps=EPS)
    return norm.rms_norm_grad(s["dy"], s["h"], s["weight"], s["dh"], eps=EPS)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------- work, exact

def work(case):
    es = torch.empty((), dtype=TYPES[case["type"]]).element_size()
    op, T = case["op"], case["T"]
    if op == "layer":
        topk, E, D, inner = case["topk"], case["E"], case["D"], case["I"]
        # experts that at least one route reaches, with evenly spread tokens
        live = E * (1.0 - (1.0 - topk / E) ** T)
        blocks = -(-2 * inner // 128) * -(-D // 128) + -(-D // 128) * -(-inner // 128)
        return {"bytes": 2 * T * D * es + E * D * es + live * (3 * inner * D + 4 * blocks),
                "flops": 2 * T * topk * 3 * inner * D + 2 * T * E * D}
    if op in ("gate", "gate_grad"):
        topk, E = case["topk"], case["E"]
        rows = 1 if op == "gate" else 2
        return {"bytes": rows * T * E * es + 8 * T * topk + (4 * E if case["bias"] else 0),
                "flops": 4 * T * E}
    D, rows = case["D"], T * case["D"]
    if op == "norm_grad":
        return {"bytes": (4 if case["residual"] else 3) * rows * es + 2 * D * es,
                "flops": 12 * rows}
    read = (2 if case["residual"] else 1) * rows * es + D * es
    kept = rows * es if case["residual"] else 0
    out = rows + 4 * T * -(-D // 128) if op == "norm_fp8" else rows * es
    return {"bytes": read + kept + out, "flops": (8 if op == "norm_fp8" else 5) * rows}


def _exact_e4m3(v):
    """v (64 bits, |v| <= 448) rounded to the nearest E4M3 value, ties to even:
    steps of 2^(exponent - 3), exponent at least -6."""
    exponent = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(exponent - 3)
    return torch.round(v / step) * step


def _exact_blocks(x):
    """Codes' values and scales [rows, blocks] of 64-bit rows."""
    q, scales = torch.empty_like(x), []
    for a in range(0, x.shape[1], 128):
        block = x[:, a:a + 128]
        amax = block.abs().amax(1, keepdim=True).clamp(min=AMAX_FLOOR)
        q[:, a:a + 128] = _exact_e4m3(block * E4M3_MAX / amax)
        scales.append(amax / E4M3_MAX)
    return q, torch.cat(scales, 1)


def _exact_values(x):
    q, scales = _exact_blocks(x)
    for b in range(scales.shape[1]):
        q[:, 128 * b:128 * b + 128] *= scales[:, b:b + 1]
    return q


def _exact_matrix(pair, e):
    codes, scales = pair[0][e].double(), pair[1][e].double()
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            codes[128 * i:128 * i + 128, 128 * j:128 * j + 128] *= scales[i, j]
    return codes


def _exact_choice(logits, s):
    """Each token's experts and weights, one after the other: the largest score (with
    the bias) that is left, the lowest number among equals."""
    if s["score"] == "sigmoid":
        scores = torch.sigmoid(logits)
    else:
        scores = torch.exp(logits - torch.logsumexp(logits, 1, keepdim=True))
    left = (logits if s["bias"] is None else scores + s["bias"].double()).clone()
    numbers = torch.arange(logits.shape[1], device=logits.device)
    ids = []
    for _ in range(s["topk"]):
        best = left.amax(1, keepdim=True)
        first = torch.where(left == best, numbers, logits.shape[1]).amin(1)
        ids.append(first)
        left[torch.arange(len(first), device=first.device), first] = -math.inf
    ids = torch.stack(ids, 1)
    chosen = scores.gather(1, ids)
    weights = chosen / chosen.sum(1, keepdim=True) if s["renormalize"] else chosen
    return ids, weights * s["scale"]


def _exact_layer(s):
    x = s["x"].double()
    ids, weights = _exact_choice(x @ s["router"].double().t(), s)
    rows = _exact_values(x)
    inner = s["down"][0].shape[2]
    out = torch.zeros_like(x)
    for e in ids.unique().tolist():
        t, k = (ids == e).nonzero(as_tuple=True)
        gu = rows[t] @ _exact_matrix(s["gate_up"], e).t()
        h = torch.nn.functional.silu(gu[:, :inner]) * gu[:, inner:]
        out[t] += weights[t, k, None] * (_exact_values(h) @ _exact_matrix(s["down"], e).t())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "layer":
        return _exact_layer(s)
    if op == "gate":
        ids, weights = _exact_choice(s["logits"].double(), s)
        return ids.to(torch.int32), weights
    if op == "gate_grad":
        logits = s["logits"].double().requires_grad_()
        if s["score"] == "sigmoid":
            scores = torch.sigmoid(logits)
        else:
            scores = torch.softmax(logits, 1)
        w = scores.gather(1, s["ids"].long())
        if s["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        return torch.autograd.grad((w * s["scale"] * s["dweights"].double()).sum(), logits)[0]
    weight = s["weight"].double()
    if op == "norm_grad":
        h = s["h"].double().requires_grad_()
        weight.requires_grad_()
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * weight
        loss = (y * s["dy"].double()).sum()
        if s["dh"] is not None:
            loss = loss + (h * s["dh"].double()).sum()
        return torch.autograd.grad(loss, (h, weight))
    h = s["x"].double()
    if s["residual"] is not None:
        # the sum as it is stored: a value of the rows' type
        h = (h + s["residual"].double()).to(s["x"].dtype).double()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * weight
    if op == "norm":
        return y if s["residual"] is None else (y, h)
    q, scales = _exact_blocks(y)
    scales = scales.t().contiguous()
    return (q, scales) if s["residual"] is None else (q, scales, h)
