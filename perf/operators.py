"""Cases that measure the token movement of an MoE layer (into expert order and
back, with gradients) and the products with block-scaled 8-bit weights.

`run` computes either the plain form of an operator (elementary torch
operations in 32 bits, rounded once at the end) or, where `own` is true, the
calls a user makes of the library.
"""
import math

import torch

own = False

#: A block of activations whose largest magnitude is below this is quantised
#: as if that were its largest magnitude, so that its scale stays a normal number.
AMAX_FLOOR = 2.0 ** -100
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # a decode batch's rows copied to their experts
        dict(name="dispatch decode", op="dispatch", T=256, topk=8, E=128, D=6144, type="bf16",
             skew=0.0, dropped=0.0),
        # training: the gradient of the tokens of a skewed prefill-sized batch
        dict(name="dispatch grad 8192", op="dispatch_grad", T=8192, topk=8, E=128, D=6144,
             type="bf16", skew=1.1, dropped=0.0),
        # one user's next token: latency
        dict(name="combine one token", op="combine", T=1, topk=8, E=128, D=6144, type="bf16",
             skew=0.0, dropped=0.0),
        # a prefill's outputs back in token order, experts over capacity drop routes
        dict(name="combine 8192", op="combine", T=8192, topk=8, E=128, D=6144, type="bf16",
             skew=1.1, dropped=0.05),
        # training of the router: rows of an odd width, 16-bit floats with dropped routes
        dict(name="combine grad odd", op="combine_grad", T=1021, topk=6, E=64, D=2047,
             type="fp16", skew=1.1, dropped=0.1),
        # training of the router: a full batch
        dict(name="combine grad 4096", op="combine_grad", T=4096, topk=8, E=128, D=6144,
             type="bf16", skew=0.0, dropped=0.0),
        # one token through a dense projection: latency and the weights' bytes
        dict(name="linear one token", op="linear", M=1, N=4096, K=6144, type="bf16"),
        # an odd batch over a ragged projection (neither N nor K a multiple of 128)
        dict(name="linear odd", op="linear", M=333, N=2056, K=1552, type="fp16"),
        # the large dense product
        dict(name="linear 8192", op="linear", M=8192, N=8192, K=8192, type="bf16"),
        # decode: 16 tokens an expert through gate_up, gathered from token order
        dict(name="experts gate_up 256", op="experts", T=256, topk=8, E=128, N=4096, K=6144,
             type="bf16", skew=0.0, gather=True),
        # decode: 64 tokens an expert through the down projection, rows in route order
        dict(name="experts down 1024", op="experts", T=1024, topk=8, E=128, N=6144, K=2048,
             type="bf16", skew=0.0, gather=False),
        # skewed prefill: some experts with thousands of tokens, some with none
        dict(name="experts prefill 8192", op="experts", T=8192, topk=8, E=128, N=4096, K=6144,
             type="bf16", skew=1.1, gather=True),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "linear", "experts"])
    kind = rng.choice(["bf16", "bf16", "fp16"] if op in ("linear", "experts")
                      else ["bf16", "bf16", "fp16", "fp32"])
    if op == "linear":
        return dict(op=op, M=_log_uniform(rng, 1, 8192), N=_log_uniform(rng, 64, 8192),
                    K=16 * _log_uniform(rng, 8, 512), type=kind)
    T = _log_uniform(rng, 1, 8192)
    topk = rng.randint(1, 8)
    E = rng.choice([8, 16, 60, 64, 96, 128])
    skew = rng.choice([0.0, 0.6, 1.1])
    if op == "experts":
        return dict(op=op, T=T, topk=topk, E=E, N=_log_uniform(rng, 128, 4096),
                    K=16 * _log_uniform(rng, 16, 384), type=kind, skew=skew,
                    gather=rng.random() < 0.6)
    D = _log_uniform(rng, 128, 6144)
    if rng.random() < 0.7:
        D = max(8, D // 8 * 8)
    return dict(op=op, T=T, topk=topk, E=E, D=D, type=kind, skew=skew,
                dropped=rng.choice([0.0, 0.0, 0.05, 0.2]))


# ------------------------------------------------------------------- inputs

def _routing(gen, T, topk, E, skew, dropped=0.0):
    """Routes of T tokens: positions in expert order [T, topk] (-1: dropped),
    each position's token and slot (-1 past the live rows), the experts' first
    positions [E + 1], and those on the host."""
    dev = "cuda"
    rank = torch.randperm(E, generator=gen, device=dev) + 1
    logp = -skew * torch.log(rank.double())
    u = torch.rand((T, E), generator=gen, device=dev, dtype=torch.float64).clamp_(1e-300, 1 - 1e-16)
    ids = torch.topk(logp - torch.log(-torch.log(u)), topk, dim=1).indices
    drop = torch.rand((T, topk), generator=gen, device=dev) < dropped
    ids = torch.where(drop, E, ids).reshape(-1)
    R = T * topk
    order = torch.argsort(ids, stable=True)
    pos = torch.empty(R, dtype=torch.int64, device=dev)
    pos[order] = torch.arange(R, device=dev)
    live = ids < E
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    offsets[1:] = torch.cumsum(torch.bincount(ids, minlength=E + 1)[:E], 0)
    row_live = torch.arange(R, device=dev) < offsets[E]
    return {
        "pos": torch.where(live, pos, -1).to(torch.int32).view(T, topk).contiguous(),
        "row_token": torch.where(row_live, order // topk, -1).to(torch.int32),
        "row_slot": torch.where(row_live, order % topk, -1).to(torch.int32),
        "offsets": offsets.to(torch.int32),
        "bounds": [int(v) for v in offsets.cpu()],
        "R": R,
    }


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
    op, kind = case["op"], case["type"]
    s = {"op": op}
    if op == "linear":
        w, ws = _weights(gen, 1, case["N"], case["K"])
        s.update(w=w[0], w_scale=ws[0], x=_normal(gen, (case["M"], case["K"]), kind))
        return s
    T, topk, E = case["T"], case["topk"], case["E"]
    s.update(_routing(gen, T, topk, E, case["skew"], case.get("dropped", 0.0)))
    R = s["R"]
    if op == "experts":
        s["w"], s["w_scale"] = _weights(gen, E, case["N"], case["K"])
        s["gather"] = case["gather"]
        s["x"] = _normal(gen, (T if case["gather"] else R, case["K"]), kind)
        return s
    D = case["D"]
    if op == "dispatch":
        s["x"] = _normal(gen, (T, D), kind)
    elif op == "dispatch_grad":
        s["dout"] = _normal(gen, (R, D), kind)
    else:
        s["y"] = _normal(gen, (R, D), kind)
        weights = torch.rand((T, topk), generator=gen, device="cuda").clamp_(1e-6).log_().neg_()
        s["weights"] = weights / weights.sum(1, keepdim=True)
        if op == "combine_grad":
            s["dout"] = _normal(gen, (T, D), kind)
    return s


# --------------------------------------------------------------- plain forms

def _plain_dispatch(s):
    live = (s["row_token"] >= 0)[:, None]
    rows = s["x"].index_select(0, s["row_token"].clamp(min=0))
    return torch.where(live, rows, torch.zeros_like(rows))


def _plain_combine(y, pos, weights):
    T, topk = pos.shape
    rows = y.index_select(0, pos.clamp(min=0).reshape(-1)).view(T, topk, -1).float()
    if weights is not None:
        rows = rows * weights[:, :, None]
    rows = torch.where((pos >= 0)[:, :, None], rows, torch.zeros_like(rows))
    return rows.sum(1).to(y.dtype)


def _plain_combine_grad(s):
    y, dout, pos, weights = s["y"], s["dout"], s["pos"], s["weights"]
    T, topk = pos.shape
    rows = y.index_select(0, pos.clamp(min=0).reshape(-1)).view(T, topk, -1).float()
    dw = (rows * dout.float()[:, None, :]).sum(2)
    dw = torch.where(pos >= 0, dw, torch.zeros_like(dw))
    token, slot = s["row_token"], s["row_slot"]
    live = (token >= 0)[:, None]
    at = token.clamp(min=0).long() * topk + slot.clamp(min=0)
    dy = dout.index_select(0, token.clamp(min=0)).float() * weights.reshape(-1)[at][:, None]
    return torch.where(live, dy, torch.zeros_like(dy)).to(y.dtype), dw


def _plain_quantise(x):
    """x as the values that its E4M3 codes and 1 x 128 scales stand for."""
    M, K = x.shape
    kb = -(-K // 128)
    blocks = torch.nn.functional.pad(x.float(), (0, kb * 128 - K)).view(M, kb, 128)
    amax = blocks.abs().amax(2, keepdim=True).clamp(min=AMAX_FLOOR)
    # x * 448 is exact for 16-bit x, and the quotient rounded to 32 bits lies on
    # the same side of every E4M3 rounding border (or on it) as the exact one
    q = (blocks * E4M3_MAX / amax).to(torch.float8_e4m3fn).float()
    return (q * (amax / E4M3_MAX)).view(M, kb * 128)[:, :K]


def _plain_weight(codes, scales):
    N, K = codes.shape
    wide = scales.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return codes.float() * wide


def _plain_linear(x, w, w_scale):
    return (_plain_quantise(x) @ _plain_weight(w, w_scale).t()).to(x.dtype)


def _plain_experts(s):
    x = s["x"]
    rows = _plain_quantise(x)
    if s["gather"]:
        rows = rows.index_select(0, s["row_token"])
    out = torch.empty((s["R"], s["w"].shape[1]), dtype=x.dtype, device=x.device)
    bounds = s["bounds"]
    for e in range(len(bounds) - 1):
        a, b = bounds[e], bounds[e + 1]
        if b > a:
            out[a:b] = rows[a:b] @ _plain_weight(s["w"][e], s["w_scale"][e]).t()
    return out


def _run_plain(s):
    op = s["op"]
    if op == "dispatch":
        return _plain_dispatch(s)
    if op == "dispatch_grad":
        return _plain_combine(s["dout"], s["pos"], None)
    if op == "combine":
        return _plain_combine(s["y"], s["pos"], s["weights"])
    if op == "combine_grad":
        return _plain_combine_grad(s)
    if op == "linear":
        return _plain_linear(s["x"], s["w"], s["w_scale"])
    return _plain_experts(s)


def _run_own(s):
    from moe_grouped_gemm_nvfp4_gb300 import fp8, tokens
    op = s["op"]
    if op == "dispatch":
        return tokens.dispatch(s["x"], s["pos"], s["offsets"])
    if op == "dispatch_grad":
        return tokens.dispatch_grad(s["dout"], s["pos"])
    if op == "combine":
        return tokens.combine(s["y"], s["pos"], s["weights"])
    if op == "combine_grad":
        return tokens.combine_grad(s["dout"], s["y"], s["pos"], s["weights"], s["offsets"])
    if op == "linear":
        return fp8.linear(s["x"], s["w"], s["w_scale"])
    return fp8.expert_linear(s["x"], s["w"], s["w_scale"], s["offsets"],
                             s["pos"] if s["gather"] else None)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------- work, exact

def work(case):
    es = torch.empty((), dtype=TYPES[case["type"]]).element_size()
    op = case["op"]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * es + N * K + 4 * -(-N // 128) * -(-K // 128) + M * N * es,
                "flops": 2 * M * N * K}
    T, topk = case["T"], case["topk"]
    R = T * topk
    if op == "experts":
        # experts that at least one route reaches, at most
        E, N, K = min(case["E"], R), case["N"], case["K"]
        rows = T if case["gather"] else R
        return {"bytes": rows * K * es + E * (N * K + 4 * -(-N // 128) * -(-K // 128))
                + R * N * es + (4 * R if case["gather"] else 0),
                "flops": 2 * R * N * K}
    D = case["D"]
    live = R * (1.0 - case["dropped"])
    if op == "dispatch":
        return {"bytes": (T + R) * D * es + 4 * R, "flops": 0}
    if op == "dispatch_grad":
        return {"bytes": (T + live) * D * es + 4 * R, "flops": live * D}
    if op == "combine":
        return {"bytes": (T + live) * D * es + 8 * R, "flops": 2 * live * D}
    return {"bytes": (T + live + R) * D * es + 12 * R, "flops": 3 * live * D}


def _exact_e4m3(v):
    """v (64 bits, |v| <= 448) rounded to the nearest E4M3 value, ties to even:
    steps of 2^(exponent - 3), exponent at least -6."""
    exponent = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(exponent - 3)
    return torch.round(v / step) * step


def _exact_rows(x):
    M, K = x.shape
    out = x.double()
    for a in range(0, K, 128):
        block = out[:, a:a + 128]
        amax = block.abs().amax(1, keepdim=True).clamp(min=AMAX_FLOOR)
        out[:, a:a + 128] = _exact_e4m3(block * E4M3_MAX / amax) * (amax / E4M3_MAX)
    return out


def _exact_weight(codes, scales):
    N, K = codes.shape
    w = codes.double()
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            w[128 * i:128 * i + 128, 128 * j:128 * j + 128] *= scales[i, j].double()
    return w


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "linear":
        return _exact_rows(s["x"]) @ _exact_weight(s["w"], s["w_scale"]).t()
    pos = s["pos"].long()
    T, topk = pos.shape
    if op == "experts":
        # FP64 runs near one TFLOP/s: the small cases only
        if 2.0 * s["R"] * case["N"] * case["K"] > 4e12:
            return None
        out = torch.zeros((s["R"], case["N"]), dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            a, b = s["bounds"][e], s["bounds"][e + 1]
            if a < b:
                rows = s["x"][s["row_token"][a:b].long()] if s["gather"] else s["x"][a:b]
                nb, kb = s["w_scale"].shape[1:]
                w = torch.zeros((nb * 128, kb * 128), dtype=torch.float64, device="cuda")
                w[:case["N"], :case["K"]] = s["w"][e].double()
                w.view(nb, 128, kb, 128).mul_(s["w_scale"][e].double()[:, None, :, None])
                out[a:b] = _exact_rows(rows) @ w[:case["N"], :case["K"]].t()
        return out
    if op == "dispatch":
        out = torch.zeros((s["R"], case["D"]), dtype=torch.float64, device="cuda")
        for k in range(topk):
            ok = pos[:, k] >= 0
            out[pos[ok, k]] = s["x"][ok].double()
        return out
    if op == "dispatch_grad":
        out = torch.zeros((T, case["D"]), dtype=torch.float64, device="cuda")
        for k in range(topk):
            ok = pos[:, k] >= 0
            out[ok] += s["dout"][pos[ok, k]].double()
        return out
    weights = s["weights"].double()
    if op == "combine":
        out = torch.zeros((T, case["D"]), dtype=torch.float64, device="cuda")
        for k in range(topk):
            ok = pos[:, k] >= 0
            out[ok] += weights[ok, k, None] * s["y"][pos[ok, k]].double()
        return out
    dout = s["dout"].double()
    dy = torch.zeros((s["R"], case["D"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros((T, topk), dtype=torch.float64, device="cuda")
    for k in range(topk):
        ok = pos[:, k] >= 0
        dy[pos[ok, k]] = weights[ok, k, None] * dout[ok]
        dw[ok, k] = (dout[ok] * s["y"][pos[ok, k]].double()).sum(1)
    return dy, dw
