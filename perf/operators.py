"""Measured cases of the beam-search decode step on int8 weights: rows quantized to
int8, the int8 product with a scale per token and per channel, the selection over
beams and vocabulary, and the reordering of the beams' states.

`own` says which side runs: the plain torch form or this library's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
F32_MAX = 3.4028234663852886e38


def listed():
    return [
        # one decoded token entering a 3584-wide projection: latency only
        {"name": "quantize-1x3584-f32", "op": "quantize", "N": 1, "K": 3584, "dtype": "f32"},
        # a prefill's activations in front of the 18944 -> 3584 down projection
        {"name": "quantize-4096x18944-bf16", "op": "quantize", "N": 4096, "K": 18944, "dtype": "bf16"},
        # q, k and v stacked, four beams of one request
        {"name": "product-4608x3584-n4-f32", "op": "product", "M": 4608, "K": 3584, "N": 4, "out": "f32", "bias": True},
        # the 152064-token head for 4 requests of 4 beams
        {"name": "product-152064x3584-n16-f32", "op": "product", "M": 152064, "K": 3584, "N": 16, "out": "f32", "bias": False},
        # the down projection for 16 requests of 4 beams: few rows, long sums
        {"name": "product-3584x18944-n64-bf16", "op": "product", "M": 3584, "K": 18944, "N": 64, "out": "bf16", "bias": False},
        # nothing a multiple of anything
        {"name": "product-5003x1001-n77-f16", "op": "product", "M": 5003, "K": 1001, "N": 77, "out": "f16", "bias": True},
        # gate and up stacked, a prefill of 4096 tokens
        {"name": "product-37888x3584-n4096-bf16", "op": "product", "M": 37888, "K": 3584, "N": 4096, "out": "bf16", "bias": False},
        # one request, four beams, twice as many candidates as beams
        {"name": "select-1x4x152064-f32", "op": "select", "B": 1, "W": 4, "V": 152064, "n": 8, "dtype": "f32", "masked": 0.0,
         "finished": False, "alpha": 0.0},
        # a full batch with finished beams and a length penalty
        {"name": "select-16x8x152064-bf16", "op": "select", "B": 16, "W": 8, "V": 152064, "n": 8, "dtype": "bf16", "masked": 0.0,
         "finished": True, "alpha": 0.8},
        # constrained decoding: most tokens masked, odd vocabulary
        {"name": "select-3x5x5003-f16", "op": "select", "B": 3, "W": 5, "V": 5003, "n": 10, "dtype": "f16", "masked": 0.9,
         "finished": True, "alpha": 1.0},
        # every layer's keys and values of one request at a short context, in place
        {"name": "reorder-56x4x37-inplace", "op": "reorder", "tensors": 56, "B": 1, "W": 4, "heads": 4, "T": 37, "Tmax": 64, "D": 128,
         "dtype": "bf16", "inplace": True},
        # eight layers' keys and values of 8 requests at 2048 tokens, into second buffers
        {"name": "reorder-16x32x2048", "op": "reorder", "tensors": 16, "B": 8, "W": 4, "heads": 4, "T": 2048, "Tmax": 2048, "D": 128,
         "dtype": "bf16", "inplace": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "select", "select", "reorder"])
    if op == "quantize":
        return {"op": op, "N": _log(rng, 1, 4096), "K": _log(rng, 32, 18944), "dtype": rng.choice(list(DTYPES))}
    if op == "product":
        M = _log(rng, 17, 152064)
        K = _log(rng, 32, min(18944, 152064 * 3584 // M))
        N = _log(rng, 1, max(1, min(4096, 37888 * 3584 * 4096 // (M * K), 37888 * 4096 // M)))
        return {"op": op, "M": M, "K": K, "N": N, "out": rng.choice(list(DTYPES)), "bias": rng.random() < 0.5}
    if op == "select":
        W = rng.choice([1, 2, 3, 4, 5, 6, 8, 10, 12, 16])
        B = _log(rng, 1, max(1, 128 // W))
        done = rng.random() < 0.5
        return {"op": op, "B": B, "W": W, "V": _log(rng, 97, 152064), "n": W if done else 2 * W, "dtype": rng.choice(list(DTYPES)),
                "masked": rng.choice([0.0, 0.0, 0.5, 0.9]), "finished": done, "alpha": rng.choice([0.0, 0.6, 1.0, 2.0])}
    W = rng.choice([2, 3, 4, 5, 8, 12])
    B = _log(rng, 1, 8)
    D = rng.choice([64, 128, 80, 33])
    T = _log(rng, 1, max(1, 32 * 2048 * 128 // (B * W * D)))
    return {"op": op, "tensors": rng.randint(1, 16), "B": B, "W": W, "heads": 4, "T": T, "Tmax": T + rng.choice([0, 1, 64]), "D": D,
            "dtype": rng.choice(list(DTYPES)) if B * W * T * D < 16 * 2048 * 128 else "bf16", "inplace": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _quantize_inputs(c, g):
    # activations after a norm or a gate: normal, a scale per token, a few channels far out
    x = torch.randn(c["N"], c["K"], generator=g, device=DEV)
    x *= torch.exp(torch.randn(c["N"], 1, generator=g, device=DEV))
    far = torch.randint(0, c["K"], (1 + c["K"] // 500,), generator=g, device=DEV)
    x[:, far] *= 12
    return {"x": x.to(DTYPES[c["dtype"]])}


def _int8(shape, g):
    return (torch.randn(shape, generator=g, device=DEV) * 40).round_().clamp_(-127, 127).to(torch.int8)


def _product_inputs(c, g):
    M, K, N = c["M"], c["K"], c["N"]
    ld = -(-K // 64) * 64  # rows of quantized activations as the quantizer leaves them: zeros up to a multiple of 64
    xq = torch.zeros(N, ld, dtype=torch.int8, device=DEV)
    xq[:, :K] = _int8((N, K), g)
    return {"w": _int8((M, K), g), "xq": xq,
            "w_scale": (torch.rand(M, generator=g, device=DEV) + 0.5) * 1e-3, "x_scale": (torch.rand(N, generator=g, device=DEV) + 0.5) * 2e-2,
            "bias": torch.randn(M, generator=g, device=DEV) if c["bias"] else None}


def _select_inputs(c, g):
    B, W, V = c["B"], c["W"], c["V"]
    z = torch.randn(B * W, V, generator=g, device=DEV) * 2.5
    z[:, torch.randint(0, V, (1 + V // 2000,), generator=g, device=DEV)] += 8  # tokens the context asks for
    z = z.to(DTYPES[c["dtype"]])
    if c["masked"]:
        off = torch.rand(B * W, V, generator=g, device=DEV) < c["masked"]
        z[off] = -math.inf
        z[0] = -math.inf  # a beam that the grammar has led nowhere
        z[B * W - 1, : V // 2] = torch.finfo(z.dtype).min  # masked by the type's lowest value
    s = {"logits": z, "score": -60 * torch.rand(B, W, generator=g, device=DEV), "finished": None, "length": None}
    if c["finished"]:
        s["finished"] = torch.rand(B, W, generator=g, device=DEV) < 0.2
    s["length"] = torch.randint(1, 200, (B, W), generator=g, device=DEV, dtype=torch.int32)
    return s


def _reorder_inputs(c, g):
    rows = c["B"] * c["W"]
    shape = (rows, c["heads"], c["Tmax"], c["D"])
    make = lambda: torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(DTYPES[c["dtype"]])  # noqa: E731
    full = [make() for _ in range(c["tensors"])]
    if c["inplace"]:
        # some beams live on, the others become copies of them: a map that leaves the same
        # rows when it is applied to its own result, as a pass repeated on one state does
        lives = torch.rand(c["B"], c["W"], generator=g, device=DEV)
        best = lives.argmax(1, keepdim=True)
        here = torch.arange(c["W"], device=DEV).expand(c["B"], -1)
        parent = torch.where(lives > 0.5, here, best)
    else:
        parent = torch.randint(0, c["W"], (c["B"], c["W"]), generator=g, device=DEV)
    cut = lambda t: t[:, :, : c["T"]]  # noqa: E731  (the tokens that are there; the rest of the buffer is room)
    return {"states": [cut(t) for t in full], "parent": parent.to(torch.int32),
            "out": None if c["inplace"] else [cut(torch.zeros_like(t)) for t in full]}


_INPUTS = {"quantize": _quantize_inputs, "product": _product_inputs, "select": _select_inputs, "reorder": _reorder_inputs}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = _INPUTS[case["op"]](case, g)
    s["case"] = case
    if own and case["op"] == "product":  # a model's weights are packed once, when they are loaded
        import quantized_gemv_argmax_amd as qg

        s["packed"] = qg.pack_i8(s["w"])
    return s


# ------------------------------------------------------------------ the plain forms
def _plain_quantize(s):
    x = s["x"].float()
    scale = (x.abs().amax(1).double() / 127).float()
    q = torch.round(x.double() / scale.double()[:, None]).clamp(-127, 127)  # a quotient next to a half decides a step
    return {"q": torch.where(scale[:, None] > 0, q, 0.0).to(torch.int8), "scale": scale}


def _plain_product(s):
    K = s["w"].shape[1]
    y = (s["xq"][:, :K].float() @ s["w"].float().t()) * (s["x_scale"][:, None] * s["w_scale"])
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(DTYPES[s["case"]["out"]])


EOS = 2


def _plain_select(s):
    c = s["case"]
    B, W, V, n = c["B"], c["W"], c["V"], c["n"]
    z = s["logits"].double().view(B, W, V).clamp(max=F32_MAX)
    z = torch.where(z.isnan(), -math.inf, z)
    top = z.amax(2, keepdim=True)
    d = torch.where(top > -math.inf, z - top, -math.inf)
    # 64 bits: the scores of two beams' candidates are compared with each other
    score = s["score"].double()[..., None] + (d - d.exp().sum(2, keepdim=True).log())
    score = torch.where(z > -math.inf, score, -math.inf)
    length = s["length"] + 1
    finished = torch.zeros(B, W, dtype=torch.bool, device=z.device)
    if s["finished"] is not None:
        finished = s["finished"]
        only = torch.full_like(score, -math.inf)
        only[:, :, EOS] = s["score"].double()
        score = torch.where(finished[..., None], only, score)
        length = torch.where(finished, s["length"], length)
    rank = score / length.double().clamp(min=1).pow(c["alpha"])[..., None]
    rank, at = torch.sort(rank.view(B, W * V), dim=1, descending=True, stable=True)  # equal: the lowest index first
    at = at[:, :n]
    there = rank[:, :n] > -math.inf
    parent, token = at // V, at % V
    return {"token": torch.where(there, token, -1).int(), "parent": torch.where(there, parent, -1).int(),
            "score": torch.where(there, score.view(B, W * V).gather(1, at), -math.inf).float(),
            "finished": there & (finished.gather(1, parent) | (token == EOS)),
            "length": torch.where(there, length.gather(1, parent), 0).int()}


def _plain_reorder(s):
    c = s["case"]
    rows = (torch.arange(c["B"], device=DEV)[:, None] * c["W"] + s["parent"]).view(-1)
    if s["out"] is None:
        return [t.copy_(t.index_select(0, rows)) for t in s["states"]]
    return [o.copy_(t.index_select(0, rows)) for t, o in zip(s["states"], s["out"])]


_PLAIN = {"quantize": _plain_quantize, "product": _plain_product, "select": _plain_select, "reorder": _plain_reorder}


# ------------------------------------------------------------------ the library's calls
def _own_quantize(s):
    import quantized_gemv_argmax_amd as qg

    q, scale = qg.quantize_i8_rows(s["x"])
    return {"q": q[:, : s["case"]["K"]], "scale": scale}


def _own_product(s):
    import quantized_gemv_argmax_amd as qg

    c = s["case"]
    y = qg.qgemm_i8(s["packed"], s["w_scale"], s["xq"], s["x_scale"], c["M"], c["K"], bias=s["bias"], dtype=DTYPES[c["out"]])
    return y[:, : c["M"]]


def _own_select(s):
    import quantized_gemv_argmax_amd as qg

    c = s["case"]
    r = qg.logits_beam_select(s["logits"], s["score"], c["n"], finished=s["finished"], length=s["length"], eos=EOS,
                              length_penalty=c["alpha"])
    return {"token": r.token, "parent": r.parent, "score": r.score, "finished": r.finished, "length": r.length}


def _own_reorder(s):
    import quantized_gemv_argmax_amd as qg

    return qg.beam_reorder(s["states"], s["parent"], out=s["out"])


_OWN = {"quantize": _own_quantize, "product": _own_product, "select": _own_select, "reorder": _own_reorder}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["N"] * case["K"]
        return {"bytes": n * (SIZES[case["dtype"]] + 1) + 4 * case["N"], "flops": 2 * n}
    if op == "product":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": M * K + N * K + 4 * (M + N) + 4 * M * case["bias"] + N * M * SIZES[case["out"]], "flops": 2 * M * K * N}
    if op == "select":
        n = case["B"] * case["W"] * case["V"]
        return {"bytes": n * SIZES[case["dtype"]] + 17 * case["B"] * (case["W"] + case["n"]), "flops": 4 * n}
    row = case["heads"] * case["T"] * case["D"] * SIZES[case["dtype"]] * case["tensors"]
    rows = case["B"] * case["W"]
    if case["inplace"]:  # about half of the beams change hands, each from its item's best one
        return {"bytes": row * (case["B"] + rows / 2), "flops": 0}
    distinct = case["B"] * case["W"] * (1 - (1 - 1 / case["W"]) ** case["W"])  # of W draws out of W
    return {"bytes": row * (rows + distinct), "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_quantize(s):
    x = s["x"].double().cpu().numpy()
    a = np.abs(x).max(1) / 127.0
    d = a.astype(np.float32).astype(np.float64)  # the scale that is stored is the one divided by
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.clip(np.rint(x / d[:, None]), -127, 127)
    q[d == 0] = 0
    return {"q": q.astype(np.int8), "scale": a}


def _exact_product(s):
    K = s["w"].shape[1]
    acc = torch.mm(s["w"].double(), s["xq"][:, :K].double().t().contiguous()).t()  # whole numbers below 2^53
    y = acc * s["w_scale"].double()[None] * s["x_scale"].double()[:, None]
    return y if s["bias"] is None else y + s["bias"].double()[None]


def _exact_select(s):
    c = s["case"]
    B, W, V, n = c["B"], c["W"], c["V"], c["n"]
    z = s["logits"].double().cpu().numpy().reshape(B, W, V)
    z = np.minimum(np.where(np.isnan(z), -np.inf, z), F32_MAX)
    cum, length = s["score"].double().cpu().numpy(), s["length"].cpu().numpy()
    done = np.zeros((B, W), bool) if s["finished"] is None else s["finished"].cpu().numpy()
    out = {"token": np.full((B, n), -1, np.int32), "parent": np.full((B, n), -1, np.int32), "score": np.full((B, n), -np.inf),
           "finished": np.zeros((B, n), bool), "length": np.zeros((B, n), np.int32)}
    for b in range(B):
        found = []  # (rank, beam, token, score, length)
        for w in range(W):
            new = int(length[b, w]) + (0 if done[b, w] else 1)
            over = float(max(new, 1)) ** c["alpha"]
            if done[b, w]:
                found.append((-cum[b, w] / over, w, EOS, cum[b, w], new))
                continue
            row = z[b, w]
            keep = np.flatnonzero(row > -np.inf)
            if not keep.size:
                continue
            d = row[keep] - row[keep].max()
            logp = d - math.log(math.fsum(np.exp(d)))
            best = keep[np.lexsort((keep, -d))[:n]] if keep.size <= 4096 else None
            if best is None:
                part = np.partition(d, d.size - n)[d.size - n]
                cand = np.flatnonzero(d >= part)
                best = keep[cand[np.lexsort((cand, -d[cand]))[:n]]]
            at = np.searchsorted(keep, best)
            found += [(-(cum[b, w] + logp[i]) / over, w, int(keep[i]), cum[b, w] + logp[i], new) for i in at]
        for j, (_, w, v, sc, new) in enumerate(sorted(found)[:n]):
            out["token"][b, j], out["parent"][b, j], out["score"][b, j], out["length"][b, j] = v, w, sc, new
            out["finished"][b, j] = done[b, w] or v == EOS
    return out


def _exact_reorder(s):
    return None  # rows are moved, nothing is computed


def exact(case, seed):
    s = _INPUTS[case["op"]](case, _seeded(seed))
    s["case"] = case
    return {"quantize": _exact_quantize, "product": _exact_product, "select": _exact_select, "reorder": _exact_reorder}[case["op"]](s)


def _seeded(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g
