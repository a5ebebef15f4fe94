"""Measured cases of a mixture-of-experts layer on 8-bit floating-point weights: rows
quantized to e4m3 with a scale per 128 values, products whose weights have a scale per
128 x 128 block, the same grouped by expert, the selection of experts and the weighted
sum of their outputs.

`own` says which side runs: the plain torch form or this library's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
F32_MAX = 3.4028234663852886e38


def listed():
    return [
        # one decoded token entering a 3584-wide projection: latency only
        {"name": "quantize-1x3584-bf16", "op": "quantize", "N": 1, "K": 3584, "dtype": "bf16", "gated": False},
        # a prefill's gate and up halves on their way into the 18944 -> 3584 down projection
        {"name": "quantize-gated-4096x18944-bf16", "op": "quantize", "N": 4096, "K": 18944, "dtype": "bf16", "gated": True},
        # q, k and v stacked, one token
        {"name": "product-4608x3584-n1-bf16", "op": "product", "M": 4608, "K": 3584, "N": 1, "out": "bf16", "bias": True},
        # gate and up stacked, a prefill of 4096 tokens
        {"name": "product-37888x3584-n4096-bf16", "op": "product", "M": 37888, "K": 3584, "N": 4096, "out": "bf16", "bias": False},
        # one token through the gate and up halves of 8 of 128 experts
        {"name": "grouped-128e8-1x2048-1536", "op": "grouped", "E": 128, "k": 8, "N": 1, "M": 1536, "K": 2048, "out": "bf16",
         "gather": True, "bias": False},
        # odd sizes everywhere, few rows to an expert
        {"name": "grouped-37e3-45x1001-517", "op": "grouped", "E": 37, "k": 3, "N": 45, "M": 517, "K": 1001, "out": "f32",
         "gather": True, "bias": True},
        # the down projections of a decode batch of 256 sequences, rows in the experts' order
        {"name": "grouped-128e8-256x768-2048", "op": "grouped", "E": 128, "k": 8, "N": 256, "M": 2048, "K": 768, "out": "bf16",
         "gather": False, "bias": False},
        # a prefill of 4096 tokens, gate and up
        {"name": "grouped-128e8-4096x2048-1536", "op": "grouped", "E": 128, "k": 8, "N": 4096, "M": 1536, "K": 2048, "out": "bf16",
         "gather": True, "bias": False},
        # the experts of a prefill's tokens
        {"name": "select-4096x128-8-f32", "op": "select", "N": 4096, "E": 128, "k": 8, "dtype": "f32", "masked": False, "normalize": True},
        # a padded decode batch with experts that are switched off
        {"name": "select-45x37-3-f16", "op": "select", "N": 45, "E": 37, "k": 3, "dtype": "f16", "masked": True, "normalize": False},
        # a prefill's outputs back in the tokens' order, onto the residual
        {"name": "combine-4096x8x2048-bf16", "op": "combine", "N": 4096, "k": 8, "M": 2048, "dtype": "bf16", "add": True, "masked": False},
        # a padded decode batch
        {"name": "combine-45x3x517-f16", "op": "combine", "N": 45, "k": 3, "M": 517, "dtype": "f16", "add": False, "masked": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "grouped", "grouped", "grouped", "select", "combine"])
    if op == "quantize":
        N, K = _log(rng, 1, 4096), _log(rng, 32, 18944)
        return {"op": op, "N": N, "K": K, "dtype": rng.choice(list(DTYPES) if N * K < 1 << 25 else ["f16", "bf16"]), "gated": rng.random() < 0.5}
    if op == "product":
        M = _log(rng, 17, 152064)
        K = _log(rng, 32, min(18944, 152064 * 3584 // M))
        N = _log(rng, 1, max(1, min(4096, 37888 * 3584 * 4096 // (M * K), 37888 * 4096 // M)))
        return {"op": op, "M": M, "K": K, "N": N, "out": rng.choice(list(DTYPES)), "bias": rng.random() < 0.5}
    if op == "grouped":
        E = rng.choice([4, 8, 16, 29, 60, 64, 128, 256])
        k = min(E, rng.choice([1, 2, 4, 6, 8]))
        M = _log(rng, 64, 4096)
        K = _log(rng, 64, max(64, min(8192, 128 * 1536 * 2048 // (E * M))))
        N = _log(rng, 1, max(1, min(4096, 32768 * 1536 * 2048 // (k * M * K), 32768 * 1536 // (k * M))))
        return {"op": op, "E": E, "k": k, "N": N, "M": M, "K": K, "out": rng.choice(list(DTYPES)), "gather": rng.random() < 0.5,
                "bias": rng.random() < 0.3}
    if op == "select":
        E = _log(rng, 2, 512)
        return {"op": op, "N": _log(rng, 1, 4096), "E": E, "k": min(E, rng.choice([1, 2, 3, 6, 8])), "dtype": rng.choice(list(DTYPES)),
                "masked": rng.random() < 0.5, "normalize": rng.random() < 0.5}
    k = rng.choice([1, 2, 3, 6, 8])
    M = _log(rng, 33, 7168)
    return {"op": op, "N": _log(rng, 1, max(1, min(4096, 32768 * 2048 // (k * M)))), "k": k, "M": M, "dtype": rng.choice(["f16", "bf16"]),
            "add": rng.random() < 0.5, "masked": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _pad(n, to):
    return -(-n // to) * to


def _quantize_inputs(c, g):
    # activations after a norm (or a gate's two halves): normal, a scale per token, a few channels far out
    W = c["K"] * (2 if c["gated"] else 1)
    x = torch.randn(c["N"], W, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(c["N"], 1, generator=g, device=DEV))
    x[:, torch.randint(0, W, (1 + W // 500,), generator=g, device=DEV)] *= 12
    return {"x": x.to(DTYPES[c["dtype"]])}


def _f8(shape, spread, g):
    return (torch.randn(shape, generator=g, device=DEV) * spread).clamp_(-F8_MAX, F8_MAX).to(F8)


def _rows(N, K, g):
    """Activations as the quantizer leaves them: rows of whole blocks, zeros beyond K, and a scale per block."""
    nb = _pad(K, 128) // 128
    xq = torch.zeros(N, nb * 128, device=DEV).to(F8)
    xq.view(torch.uint8)[:, :K] = _f8((N, K), 150, g).view(torch.uint8)
    return xq, (torch.rand(N, _pad(nb, 4), generator=g, device=DEV) + 0.5) * 4e-3


def _bias(shape, given, g):
    return torch.randn(shape, generator=g, device=DEV) if given else None


def _product_inputs(c, g):
    M, K, N = c["M"], c["K"], c["N"]
    xq, xs = _rows(N, K, g)
    return {"w": _f8((M, K), 110, g), "w_scale": (torch.rand(-(-M // 128), -(-K // 128), generator=g, device=DEV) + 0.5) * 2e-4,
            "xq": xq, "x_scale": xs, "bias": _bias(M, c["bias"], g)}


def _experts_of(N, E, k, g):
    """Distinct experts of each token, some asked for more often than others."""
    z = torch.randn(N, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
    return z.topk(k, dim=1).indices


def _grouped_inputs(c, g):
    E, k, N, M, K = c["E"], c["k"], c["N"], c["M"], c["K"]
    flat, order = torch.sort(_experts_of(N, E, k, g).reshape(-1), stable=True)
    offsets = torch.searchsorted(flat, torch.arange(E + 1, device=DEV)).to(torch.int32)
    xq, xs = _rows(N if c["gather"] else N * k, K, g)
    ends = offsets.tolist()  # the plain form walks the experts on the host
    return {"w": _f8((E, M, K), 110, g), "w_scale": (torch.rand(E, -(-M // 128), -(-K // 128), generator=g, device=DEV) + 0.5) * 2e-4,
            "xq": xq, "x_scale": xs, "bias": _bias((E, M), c["bias"], g), "offsets": offsets,
            "row": (order // k).to(torch.int32) if c["gather"] else None,
            "parts": [(e, ends[e], ends[e + 1]) for e in range(E) if ends[e + 1] > ends[e]]}


def _select_inputs(c, g):
    N, E = c["N"], c["E"]
    z = torch.randn(N, E, generator=g, device=DEV) * 1.5 + 0.5 * torch.randn(E, generator=g, device=DEV)
    z = z.to(DTYPES[c["dtype"]])
    if c["masked"]:
        z[:, torch.rand(E, generator=g, device=DEV) < 0.2] = -math.inf  # experts switched off
        z[torch.rand(N, generator=g, device=DEV) < 0.1] = -math.inf  # padding among the tokens
        z[N - 1] = -math.inf
        z[0, : E // 2] = torch.finfo(z.dtype).min  # masked by the type's lowest value
    return {"logits": z}


def _combine_inputs(c, g):
    N, k, M = c["N"], c["k"], c["M"]
    R = N * k
    position = torch.randperm(R, generator=g, device=DEV).view(N, k).to(torch.int32)
    if c["masked"]:
        position[torch.rand(N, k, generator=g, device=DEV) < 0.2] = -1
        position[N - 1] = -1
    w = torch.rand(N, k, generator=g, device=DEV)
    t = DTYPES[c["dtype"]]
    return {"y": torch.randn(R, M, generator=g, device=DEV).to(t), "position": position, "weight": w / w.sum(1, keepdim=True),
            "add": torch.randn(N, M, generator=g, device=DEV).to(t) if c["add"] else None}


_INPUTS = {"quantize": _quantize_inputs, "product": _product_inputs, "grouped": _grouped_inputs, "select": _select_inputs,
           "combine": _combine_inputs}


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = _INPUTS[case["op"]](case, g)
    s["case"] = case
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] in ("product", "grouped"):  # a model's weights are packed once, when they are loaded
        import quantized_gemv_argmax_amd as qg

        s["packed"] = qg.pack_f8(s["w"])
    return s


# ------------------------------------------------------------------ the plain forms
def _plain_quantize(s):
    c = s["case"]
    N, K = c["N"], c["K"]
    x = s["x"].float()
    if c["gated"]:
        x = x[:, :K] / (1 + torch.exp(-x[:, :K])) * x[:, K:]
    kp = _pad(K, 128)
    x = torch.nn.functional.pad(x, (0, kp - K)).view(N, kp // 128, 128)
    scale = (x.abs().amax(2).double() / F8_MAX).float()
    t = x.double() / scale.double()[..., None]  # 64 bits: a quotient next to a border decides a step
    step = torch.ldexp(torch.ones_like(t), torch.frexp(t)[1].clamp(min=-5) - 4)
    q = (torch.round(t / step) * step).clamp(-F8_MAX, F8_MAX)
    q = torch.where(scale[..., None] > 0, q, 0.0).to(F8)
    return {"q": q.view(N, kp)[:, :K], "scale": scale}


def _values(xq, xs):
    N, kp = xq.shape
    return (xq.float().view(N, kp // 128, 128) * xs[:, : kp // 128, None]).view(N, kp)


def _weights(w, ws):
    M, K = w.shape
    return w.float() * ws.repeat_interleave(128, 0)[:M].repeat_interleave(128, 1)[:, :K]


def _plain_product(s):
    c = s["case"]
    y = _values(s["xq"], s["x_scale"])[:, : c["K"]] @ _weights(s["w"], s["w_scale"]).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(DTYPES[c["out"]])


def _plain_grouped(s):
    c = s["case"]
    x = _values(s["xq"], s["x_scale"])[:, : c["K"]]
    if s["row"] is not None:
        x = x[s["row"]]
    y = torch.empty(c["N"] * c["k"], c["M"], device=DEV, dtype=DTYPES[c["out"]])
    for e, a, b in s["parts"]:
        part = x[a:b] @ _weights(s["w"][e], s["w_scale"][e]).t()
        y[a:b] = part if s["bias"] is None else part + s["bias"][e]
    return y


def _plain_select(s):
    c = s["case"]
    N, E, k = c["N"], c["E"], c["k"]
    z = s["logits"].float().clamp(max=F32_MAX)
    z = torch.where(z.isnan(), -math.inf, z)
    best, at = torch.sort(z, dim=1, descending=True, stable=True)  # equal: the lowest index first
    there = best[:, :k] > -math.inf
    p = torch.where(best > -math.inf, torch.exp(best - best[:, :1]), 0.0)
    weight = torch.where(there, p[:, :k], 0.0)
    total = weight.sum(1, keepdim=True) if c["normalize"] else p.sum(1, keepdim=True)
    expert = torch.where(there, at[:, :k], -1)
    flat, order = torch.sort(torch.where(there, expert, E).view(-1), stable=True)
    position = torch.empty_like(order)
    position[order] = torch.arange(N * k, device=DEV)
    return {"expert": expert.int(), "weight": torch.where(there, weight / total, 0.0),
            "position": torch.where(there, position.view(N, k), -1).int(), "row": torch.where(flat < E, order // k, -1).int(),
            "offsets": torch.searchsorted(flat, torch.arange(E + 1, device=DEV)).int()}


def _plain_combine(s):
    c = s["case"]
    there = s["position"] >= 0
    y = s["y"].float()[s["position"].clamp(min=0).view(-1)].view(c["N"], c["k"], c["M"])
    y = torch.where(there[..., None], y * s["weight"][..., None], 0.0).sum(1)
    if s["add"] is not None:
        y = y + s["add"].float()
    return y.to(DTYPES[c["dtype"]])


_PLAIN = {"quantize": _plain_quantize, "product": _plain_product, "grouped": _plain_grouped, "select": _plain_select,
          "combine": _plain_combine}


# ------------------------------------------------------------------ the library's calls
def _own_quantize(s):
    import quantized_gemv_argmax_amd as qg

    K = s["case"]["K"]
    q, scale = qg.quantize_f8_rows(s["x"], gated=s["case"]["gated"])
    return {"q": q[:, :K], "scale": scale[:, : -(-K // 128)]}


def _own_product(s):
    import quantized_gemv_argmax_amd as qg

    c = s["case"]
    y = qg.qgemm_f8(s["packed"], s["w_scale"], s["xq"], s["x_scale"], c["M"], c["K"], bias=s["bias"], dtype=DTYPES[c["out"]])
    return y[:, : c["M"]]


def _own_grouped(s):
    import quantized_gemv_argmax_amd as qg

    c = s["case"]
    y = qg.qgemm_f8_grouped(s["packed"], s["w_scale"], s["xq"], s["x_scale"], c["M"], c["K"], s["offsets"], row=s["row"],
                            bias=s["bias"], dtype=DTYPES[c["out"]])
    return y[:, : c["M"]]


def _own_select(s):
    import quantized_gemv_argmax_amd as qg

    r = qg.logits_expert_select(s["logits"], s["case"]["k"], normalize=s["case"]["normalize"])
    return {"expert": r.expert, "weight": r.weight, "position": r.position, "row": r.row, "offsets": r.offsets}


def _own_combine(s):
    import quantized_gemv_argmax_amd as qg

    return qg.expert_combine(s["y"], s["position"], s["weight"], add=s["add"])


_OWN = {"quantize": _own_quantize, "product": _own_product, "grouped": _own_grouped, "select": _own_select, "combine": _own_combine}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["N"] * case["K"]
        return {"bytes": n * (SIZES[case["dtype"]] * (2 if case["gated"] else 1) + 1) + 4 * case["N"] * -(-case["K"] // 128),
                "flops": (8 if case["gated"] else 2) * n}
    if op == "product":
        M, K, N = case["M"], case["K"], case["N"]
        nb = -(-K // 128)
        return {"bytes": M * K + N * K + 4 * nb * (-(-M // 128) + N) + 4 * M * case["bias"] + N * M * SIZES[case["out"]],
                "flops": 2 * M * K * N}
    if op == "grouped":
        E, k, N, M, K = (case[n] for n in ("E", "k", "N", "M", "K"))
        used = E * (1 - (1 - k / E) ** N)  # experts that some token asks for, about
        nb = -(-K // 128)
        return {"bytes": used * (M * K + 4 * nb * -(-M // 128) + 4 * M * case["bias"]) + N * (1 if case["gather"] else k) * (K + 4 * nb)
                + 4 * (E + 1) + N * k * (M * SIZES[case["out"]] + 4 * case["gather"]), "flops": 2 * N * k * M * K}
    if op == "select":
        N, E, k = case["N"], case["E"], case["k"]
        return {"bytes": N * E * SIZES[case["dtype"]] + 16 * N * k + 4 * (E + 1), "flops": 4 * N * E}
    N, k, M = case["N"], case["k"], case["M"]
    there = 0.8 if case["masked"] else 1.0
    return {"bytes": (N * k * there + N + N * case["add"]) * M * SIZES[case["dtype"]] + 8 * N * k, "flops": 2 * N * k * M}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_quantize(s):
    c = s["case"]
    N, K = c["N"], c["K"]
    # the values that eight bits can hold, by exponent and three more bits, and the borders between them
    held = torch.tensor([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:-1],
                        dtype=torch.float64, device=DEV)
    border = (held[1:] + held[:-1]) / 2
    q, scales = torch.empty(N, K, dtype=torch.float64, device=DEV), torch.empty(N, -(-K // 128), dtype=torch.float64, device=DEV)
    for n0 in range(0, N, 512):
        x = s["x"][n0 : n0 + 512].double()
        if c["gated"]:
            x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
        for b in range(-(-K // 128)):
            block = x[:, 128 * b : 128 * b + 128].contiguous()
            d = block.abs().amax(1) / F8_MAX
            scales[n0 : n0 + 512, b] = d
            a = (block.abs() / d.float().double()[:, None]).nan_to_num(0.0).clamp(max=F8_MAX)
            i = torch.bucketize(a, border)
            i = i + ((i < 126) & (border[i.clamp(max=125)] == a) & (i % 2 == 1)).long()  # ties to the even one
            q[n0 : n0 + 512, 128 * b : 128 * b + 128] = held[i] * block.sign()
    return {"q": q, "scale": scales}


def _by_blocks(xq, xs, w, ws):
    M, K = w.shape
    y = torch.zeros(xq.shape[0], M, dtype=torch.float64, device=DEV)
    for b in range(-(-K // 128)):
        cut = slice(128 * b, min(K, 128 * b + 128))
        part = torch.mm(xq[:, cut].double(), w[:, cut].double().t().contiguous())  # whole multiples of 2^-18, below 2^53 of them
        y += part * xs[:, b].double()[:, None] * ws[:, b].double().repeat_interleave(128)[None, :M]
    return y


def _exact_product(s):
    y = _by_blocks(s["xq"], s["x_scale"], s["w"], s["w_scale"])
    return y if s["bias"] is None else y + s["bias"].double()


def _exact_grouped(s):
    c = s["case"]
    y = torch.empty(c["N"] * c["k"], c["M"], dtype=torch.float64, device=DEV)
    ends = s["offsets"].cpu().numpy()
    for e in np.flatnonzero(np.diff(ends)):
        rows = torch.arange(int(ends[e]), int(ends[e + 1]), device=DEV)
        of = rows if s["row"] is None else s["row"][rows].long()
        # (gathered by their bytes)
        part = _by_blocks(s["xq"].view(torch.uint8)[of].view(F8), s["x_scale"][of], s["w"][int(e)], s["w_scale"][int(e)])
        y[rows] = part if s["bias"] is None else part + s["bias"][int(e)].double()
    return y


def _exact_select(s):
    c = s["case"]
    N, E, k = c["N"], c["E"], c["k"]
    z = s["logits"].double().cpu().numpy()
    z = np.minimum(np.where(np.isnan(z), -np.inf, z), F32_MAX)
    expert, position = np.full((N, k), -1, np.int32), np.full((N, k), -1, np.int32)
    weight = np.zeros((N, k))
    asked = [[] for _ in range(E)]  # the (token, choice) pairs of each expert, in the tokens' order
    for n in range(N):
        keep = np.flatnonzero(z[n] > -np.inf)
        if not keep.size:
            continue
        best = keep[np.lexsort((keep, -z[n, keep]))][:k]
        p = np.exp(z[n, best] - z[n, best[0]])
        over = p.sum() if c["normalize"] else np.exp(z[n, keep] - z[n, best[0]]).sum()
        expert[n, : best.size], weight[n, : best.size] = best, p / over
        for j, e in enumerate(best):
            asked[e].append((n, j))
    row, offsets = np.full(N * k, -1, np.int32), np.zeros(E + 1, np.int32)
    at = 0
    for e in range(E):
        for n, j in asked[e]:
            position[n, j], row[at] = at, n
            at += 1
        offsets[e + 1] = at
    return {"expert": expert, "weight": weight, "position": position, "row": row, "offsets": offsets}


def _exact_combine(s):
    c = s["case"]
    y = torch.zeros(c["N"], c["M"], dtype=torch.float64, device=DEV) if s["add"] is None else s["add"].double()
    for j in range(c["k"]):
        n = torch.nonzero(s["position"][:, j] >= 0)[:, 0]
        y[n] += s["y"][s["position"][n, j].long()].double() * s["weight"][n, j].double()[:, None]
    return y


def exact(case, seed):
    s = _inputs(case, seed)
    return {"quantize": _exact_quantize, "product": _exact_product, "grouped": _exact_grouped, "select": _exact_select,
            "combine": _exact_combine}[case["op"]](s)
