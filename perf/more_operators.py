"""Cases for the operators of a layer trained and served in 8-bit floating point with a
scale for each block of 128: routing to experts with its gradient, quantisation of rows,
of weights and along a group's rows, and the gradient of the expert weights.

`run` computes a case either in its plain form (elementary torch operations in 32 bits,
the choice of experts in 64) or, where `own` is true, through the library's entry points.
Sizes are those of the library's named workloads (decode, prefill) or generic.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ITEM = {"bf16": 2, "fp16": 2, "fp32": 4}
DEV = "cuda"
BLOCK = 128          # elements that share a scale
TOP = 448.0          # the largest e4m3 value


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One token of a serving loop to its 8 of 64 experts: the smallest call, all latency.
        dict(name="route_one", op="route", tokens=1, experts=64, top_k=8, dtype="bf16", scoring="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renormalise=True, scale=1.0),
        # A decode step's 256 tokens, sigmoid scores with a balancing bias, 4 of 8 groups.
        dict(name="route_decode", op="route", tokens=256, experts=256, top_k=8, dtype="fp32", scoring="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renormalise=True, scale=2.5),
        # A prefill batch, softmax scores, the chosen weights renormalised.
        dict(name="route_prefill", op="route", tokens=32768, experts=128, top_k=8, dtype="bf16", scoring="softmax",
             bias=False, groups=1, top_groups=1, group_top=1, renormalise=True, scale=1.0),
        # Training, weights not renormalised: the gradient reaches every expert's logit.
        dict(name="route_grad_softmax", op="route_grad", tokens=16384, experts=64, top_k=6, dtype="bf16",
             scoring="softmax", renormalise=False, scale=1.0),
        # Training with renormalised sigmoid scores, an odd number of tokens and of experts.
        dict(name="route_grad_sigmoid", op="route_grad", tokens=5003, experts=161, top_k=8, dtype="fp32",
             scoring="sigmoid", renormalise=True, scale=2.5),
        # A decode step's activations, quantised while they are gathered by expert.
        dict(name="quantize_decode", op="quantize", tokens=256, top_k=8, experts=64, rows=2048, width=2048, dtype="bf16",
             skew=1.1, pow2=False),
        # The weights of a layer after an optimizer step, a scale for each 128 x 128 tile.
        dict(name="quantize_weights", op="tiles", experts=64, n=2816, k=2048, dtype="bf16", pow2=True),
        # Training, prefill shapes: the rows for the product, and along each expert's rows for the weight gradient.
        dict(name="quantize_cols_prefill", op="cols", tokens=0, top_k=1, experts=8, rows=32768, width=4096, dtype="bf16",
             skew=0.0, both=True),
        # A small fp32 step gathered from odd numbers of tokens, many experts of uneven load.
        dict(name="quantize_cols_odd", op="cols", tokens=1003, top_k=6, experts=64, rows=6018, width=1424, dtype="fp32",
             skew=1.1, both=False),
        # A small layer's weight gradient: 88 tiles at most, latency and the gradient's bytes.
        dict(name="weight_grad_small", op="weight_grad", rows=1201, experts=16, n=1024, k=512, out="fp32", skew=1.0),
        # The decode shapes' layer in training: bound by the gradient's 1.5 GB in 32 bits.
        dict(name="weight_grad_many", op="weight_grad", rows=16384, experts=64, n=2816, k=2048, out="fp32", skew=1.1),
        # The prefill shapes: bound by the tensor cores.
        dict(name="weight_grad_prefill", op="weight_grad", rows=32768, experts=8, n=14336, k=4096, out="bf16", skew=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """An odd multiple of 16, 64 or 128, spread over the logarithm of lo .. hi."""
    step = rng.choice((16, 64, 128))
    return step * (max(1, min(hi // step - 1, _log(rng, max(1.0, lo / step), hi / step))) | 1)


def draw(rng):
    op = rng.choice(("route", "route_grad", "quantize", "tiles", "cols", "weight_grad"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op in ("route", "route_grad"):
        groups = rng.choice((1, 1, 4, 8)) if op == "route" else 1
        experts = groups * max(4, _log(rng, 8, 512) // groups)
        top_groups = max(1, groups // 2)
        top_k = min(rng.choice((1, 2, 4, 6, 8)), experts // groups * top_groups)
        tokens = _log(rng, 1, min(32768, 4_000_000 // experts)) | 1
        case = dict(op=op, tokens=tokens, experts=experts, top_k=top_k, dtype=dtype,
                    scoring=rng.choice(("softmax", "sigmoid")), renormalise=rng.random() < 0.6,
                    scale=rng.choice((1.0, 2.5)))
        if op == "route_grad" and top_k == 1:
            case["renormalise"] = False      # one weight that is always 1 has no gradient
        if op == "route":
            case.update(bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, group_top=rng.choice((1, 2)))
        return case
    if op == "tiles":
        n, k = _width(rng, 128, 8192), _width(rng, 128, 8192)
        return dict(op=op, experts=max(1, min(_log(rng, 1, 64), 300_000_000 // (n * k))), n=n, k=k, dtype=dtype,
                    pow2=rng.random() < 0.5)
    experts, skew = _log(rng, 1, 128), rng.choice((0.0, 1.0, 1.1))
    if op == "weight_grad":
        n, k = _width(rng, 128, 8192), _width(rng, 128, 4096)
        experts = max(1, min(experts, 300_000_000 // (n * k)))
        rows = _log(rng, 1, max(2, min(32768, int(1.5e12 / (n * k))))) | 1
        return dict(op=op, rows=rows, experts=experts, n=n, k=k, out=rng.choice(("fp32", "bf16")), skew=skew)
    width = _width(rng, 64, 8192)
    rows = _log(rng, 1, min(32768, 100_000_000 // width)) | 1
    top_k = min(experts, rng.choice((1, 1, 2, 8)))
    tokens = 0
    if top_k > 1:
        tokens = max(1, rows // top_k)
        rows = tokens * top_k
    case = dict(op=op, tokens=tokens, top_k=top_k, experts=experts, rows=rows, width=width, dtype=dtype, skew=skew)
    case["pow2" if op == "quantize" else "both"] = rng.random() < 0.5
    return case


def work(case):
    op = case["op"]
    if op in ("route", "route_grad"):
        t, e, k, es = case["tokens"], case["experts"], case["top_k"], ITEM[case["dtype"]]
        if op == "route":
            return {"bytes": t * e * es + 8 * t * k + (4 * e if case["bias"] else 0), "flops": 4.0 * t * e}
        read = t * k if case["renormalise"] or case["scoring"] == "sigmoid" else t * e
        return {"bytes": read * es + t * e * es + 8 * t * k, "flops": 4.0 * t * e}
    if op == "tiles":
        e, n, k = case["experts"], case["n"], case["k"]
        return {"bytes": e * n * k * (ITEM[case["dtype"]] + 1) + 4 * e * -(-n // BLOCK) * -(-k // BLOCK),
                "flops": 2.0 * e * n * k}
    if op == "weight_grad":
        r, e, n, k = case["rows"], case["experts"], case["n"], case["k"]
        return {"bytes": r * (n + k) * (1 + 1 / BLOCK) + e * n * k * ITEM[case["out"]], "flops": 2.0 * r * n * k}
    r, w = case["rows"], case["width"]
    read = (case["tokens"] or r) * w * ITEM[case["dtype"]] + (4 * r if case["tokens"] else 0)
    by_row, by_col = r * w * (1 + 4 / BLOCK), r * w * (1 + 1 / BLOCK)
    if op == "quantize":
        return {"bytes": read + by_row, "flops": 2.0 * r * w}
    return {"bytes": read + by_col + (by_row if case["both"] else 0), "flops": 2.0 * r * w}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _activations(shape, g, dtype):
    """Normal values with a few channels an order of magnitude above the rest."""
    x = torch.randn(shape, generator=g, device=DEV)
    x *= torch.where(torch.rand(shape[1], generator=g, device=DEV) < 0.02, 12.0, 1.0)
    return x.to(DTYPES[dtype])


def _logits(case, g):
    """A router's logits: normal, some experts more popular than others."""
    x = 1.5 * torch.randn((case["tokens"], case["experts"]), generator=g, device=DEV)
    x += 0.7 * torch.randn(case["experts"], generator=g, device=DEV)
    return x.to(DTYPES[case["dtype"]])


def _loads(case, seed):
    rng = np.random.default_rng([int(seed), 7])
    p = np.arange(1, case["experts"] + 1, dtype=np.float64) ** -case["skew"]
    return rng.multinomial(case["rows"], p / p.sum())


def _offsets(loads):
    return torch.tensor(np.concatenate([[0], np.cumsum(loads)]), dtype=torch.int32, device=DEV)


def _pitch(rows, groups):
    """Columns of a matrix quantised along the rows: each group starts a block of 128."""
    return (rows // BLOCK + groups) * BLOCK


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("route", "route_grad"):
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        s["logits"] = _logits(case, g)
        if op == "route":
            # A bias that small steps have moved, as balancing does.
            s["bias"] = (50 * torch.randn(e, generator=g, device=DEV)).round() * 0.001 if case["bias"] else None
            s["slot_experts"] = torch.zeros((t, k), dtype=torch.int32, device=DEV)
            s["weights"] = torch.zeros((t, k), device=DEV)
        else:
            s["slot_experts"] = s["logits"].float().topk(k, dim=1).indices.to(torch.int32)
            s["d_weights"] = torch.randn((t, k), generator=g, device=DEV)
            s["d_logits"] = torch.zeros_like(s["logits"])
        return s
    if op == "tiles":
        e, n, k = case["experts"], case["n"], case["k"]
        s["w"] = torch.empty((e, n, k), dtype=DTYPES[case["dtype"]], device=DEV)
        for i in range(e):
            s["w"][i] = torch.randn((n, k), generator=g, device=DEV) * 0.02
        s["q"] = torch.zeros((e, n, k), dtype=torch.uint8, device=DEV)
        s["scales"] = torch.zeros((e, -(-n // BLOCK), -(-k // BLOCK)), device=DEV)
        return s
    loads = _loads(case, seed)
    s["a_offsets"] = _offsets(loads)
    r, e = case["rows"], case["experts"]
    p = _pitch(r, e)
    if op == "weight_grad":
        n, k = case["n"], case["k"]
        s["loads"] = [int(x) for x in loads]
        at = _columns(s["a_offsets"], r)
        s["a_t"], s["a_t_scales"] = _encode_cols(_activations((r, k), g, "fp32"), at, p)
        # Gradients of a mean over tokens: small.
        s["d_t"], s["d_t_scales"] = _encode_cols(torch.randn((r, n), generator=g, device=DEV) * 1e-4, at, p)
        s["d_b"] = torch.zeros((e, n, k), dtype=DTYPES[case["out"]], device=DEV)
        return s
    w = case["width"]
    s["x"] = _activations((case["tokens"] or r, w), g, case["dtype"])
    s["row_slots"] = torch.randperm(r, generator=g, device=DEV).to(torch.int32) if case["tokens"] else None
    rows = op == "quantize" or case["both"]
    s["q"] = torch.zeros((r, w), dtype=torch.uint8, device=DEV) if rows else None
    s["scales"] = torch.zeros((r, -(-w // BLOCK)), device=DEV) if rows else None
    if op == "cols":
        s["q_t"] = torch.zeros((w, p), dtype=torch.uint8, device=DEV)
        s["t_scales"] = torch.zeros((p // BLOCK, w), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

def _route(s):
    """Expert ids and weights.  What is compared is compared in 64 bits: two scores may be nearer than 32 hold."""
    case, t, e = s["case"], s["case"]["tokens"], s["case"]["experts"]
    x = s["logits"].double()
    score = _scores(x, case["scoring"])
    key = score + s["bias"].double() if case["bias"] else score
    if case["groups"] > 1:
        by_group = key.reshape(t, case["groups"], -1).sort(dim=2, descending=True).values[:, :, : case["group_top"]].sum(2)
        chosen = by_group.sort(dim=1, descending=True, stable=True).indices[:, : case["top_groups"]]
        keep = torch.zeros((t, case["groups"]), dtype=torch.bool, device=DEV)
        keep[torch.arange(t, device=DEV)[:, None], chosen] = True
        key = torch.where(keep.repeat_interleave(e // case["groups"], 1), key, -math.inf)
    # Equal keys go to the lowest expert.  Without a bias the logits stand in the order of their scores.
    order = key if case["bias"] else torch.where(key == -math.inf, key, x)
    ids = order.sort(dim=1, descending=True, stable=True).indices[:, : case["top_k"]]
    w = _scores(s["logits"].float(), case["scoring"]).gather(1, ids)
    if case["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    return {"slot_experts": ids.to(torch.int32), "weights": w * case["scale"]}


def _scores(x, scoring):
    if scoring == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    p = torch.exp(x - x.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def _route_grad(s):
    case = s["case"]
    ids, g = s["slot_experts"].long(), s["d_weights"] * case["scale"]
    score = _scores(s["logits"].float(), case["scoring"])
    picked = score.gather(1, ids)
    if case["renormalise"]:
        share = picked / picked.sum(1, keepdim=True)
        g = share * (g - (g * share).sum(1, keepdim=True))
        d = torch.zeros_like(score).scatter(1, ids, g * (1 - picked) if case["scoring"] == "sigmoid" else g)
    elif case["scoring"] == "sigmoid":
        d = torch.zeros_like(score).scatter(1, ids, g * picked * (1 - picked))
    else:
        d = score * (torch.zeros_like(score).scatter(1, ids, g) - (g * picked).sum(1, keepdim=True))
    return {"d_logits": d.to(s["logits"].dtype)}


def _ceil_power(amax):
    """The exponent of the smallest power of two that is at least amax / 448, from -127 up."""
    m, ex = torch.frexp(amax)
    return torch.where(m <= 0.875, ex - 9, ex - 8).clamp(min=-127)


def _power_of_two(ex):
    code = ex + 127
    return torch.where(code == 0, 0x00400000, code << 23).to(torch.int32).view(torch.float32)


def _block_scale(amax, pow2):
    """fp32 scales of blocks with these largest magnitudes; 0 for a block of zeros."""
    s = _power_of_two(_ceil_power(amax)) if pow2 else amax / TOP
    return torch.where(amax == 0, 0.0, s)


def _e4m3(x, scale):
    y = torch.where(scale == 0, 0.0, x / torch.where(scale == 0, 1.0, scale))
    return y.clamp(-TOP, TOP).to(torch.float8_e4m3fn)


def _padded(x, rows, cols):
    out = torch.zeros((rows, cols), dtype=torch.float32, device=DEV)
    out[: x.shape[0], : x.shape[1]] = x
    return out


def _quantize_rows(x, pow2):
    r, w = x.shape
    blocks = _padded(x, r, -(-w // BLOCK) * BLOCK).reshape(r, -1, BLOCK)
    scale = _block_scale(blocks.abs().amax(2), pow2)
    return _e4m3(blocks, scale[:, :, None]).reshape(r, -1)[:, :w].contiguous(), scale


def _quantize_tiles(w, pow2):
    """Weights [experts, n, k], a scale for each 128 x 128 of an expert's."""
    e, n, k = w.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    tiles = torch.zeros((e, nb * BLOCK, kb * BLOCK), dtype=torch.float32, device=DEV)
    tiles[:, :n, :k] = w
    tiles = tiles.reshape(e, nb, BLOCK, kb, BLOCK)
    scale = _block_scale(tiles.abs().amax(dim=(2, 4)), pow2)
    q = _e4m3(tiles, scale[:, :, None, :, None]).reshape(e, nb * BLOCK, -1)
    return q[:, :n, :k].contiguous(), scale


def _columns(a_offsets, rows):
    """Where each row stands in a matrix quantised along the rows."""
    r = torch.arange(rows, device=DEV, dtype=torch.int32)
    off = a_offsets.long()
    g = torch.searchsorted(a_offsets, r, right=True) - 1
    return (off[g] // BLOCK + g) * BLOCK + (r - off[g])


def _encode_cols(x, at, pitch):
    """e4m3 [width, pitch] and exponent codes [pitch / 128, width]: a scale for each 128 rows of a group."""
    full = torch.zeros((pitch, x.shape[1]), device=DEV)
    full[at] = x.float()
    blocks = full.reshape(pitch // BLOCK, BLOCK, -1)
    amax = blocks.abs().amax(1)
    ex = torch.where(amax == 0, -127, _ceil_power(amax))
    q = (blocks / _power_of_two(ex)[:, None, :]).to(torch.float8_e4m3fn)
    return q.reshape(pitch, -1).t().contiguous().view(torch.uint8), (ex + 127).to(torch.uint8)


def _decode_cols(q_t, t_scales):
    scale = _power_of_two(t_scales.to(torch.int32) - 127)
    return q_t.view(torch.float8_e4m3fn).float() * scale.t().repeat_interleave(BLOCK, 1)


def _gathered(s):
    if s["row_slots"] is None:
        return s["x"]
    return s["x"][s["row_slots"].long() // s["case"]["top_k"]]


def _values(q, scales, q_t=None, t_scales=None):
    """8-bit buffers as the values that they stand for."""
    out = {}
    if q is not None:
        out.update(q=q.view(torch.float8_e4m3fn), scales=scales)
    if q_t is not None:
        out.update(q_t=q_t.view(torch.float8_e4m3fn), t_scales=t_scales.view(torch.float8_e8m0fnu))
    return out


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "route":
        return _route(s)
    if op == "route_grad":
        return _route_grad(s)
    if op == "quantize":
        return _values(*_quantize_rows(_gathered(s).float(), case["pow2"]))
    if op == "tiles":
        return _values(*_quantize_tiles(s["w"], case["pow2"]))
    if op == "cols":
        x = _gathered(s).float()
        rows = _quantize_rows(x, False) if case["both"] else (None, None)
        return _values(*rows, *_encode_cols(x, _columns(s["a_offsets"], case["rows"]), s["q_t"].shape[1]))
    a, d = _decode_cols(s["a_t"], s["a_t_scales"]), _decode_cols(s["d_t"], s["d_t_scales"])
    out = torch.empty_like(s["d_b"])
    first = 0
    for i, load in enumerate(s["loads"]):
        c = (first // BLOCK + i) * BLOCK
        out[i] = d[:, c:c + load] @ a[:, c:c + load].t()
        first += load
    return {"d_b": out}


# ---------------------------------------------------------------- the library's calls

_handles = {}


def _handle(experts):
    """The handle that a program keeps for its number of experts."""
    from ragged_matmul_gb300 import binding
    if experts not in _handles:
        _handles[experts] = binding.gmm_create(experts, torch.cuda.current_device())
    return _handles[experts]


def _library(s):
    from ragged_matmul_gb300 import binding
    case, op = s["case"], s["case"]["op"]
    h = _handle(case["experts"])
    if op == "route":
        binding.gmm_route(h, s["slot_experts"], s["weights"], s["logits"], scoring=case["scoring"], bias=s["bias"],
                          expert_groups=case["groups"], top_groups=case["top_groups"], group_top=case["group_top"],
                          renormalise=case["renormalise"], scale=case["scale"])
        return {"slot_experts": s["slot_experts"], "weights": s["weights"]}
    if op == "route_grad":
        binding.gmm_route_grad(h, s["d_logits"], s["d_weights"], s["slot_experts"], s["logits"],
                               scoring=case["scoring"], renormalise=case["renormalise"], scale=case["scale"])
        return {"d_logits": s["d_logits"]}
    if op == "quantize":
        binding.gmm_quantize_fp8(h, s["q"], s["scales"], s["x"], row_slots=s["row_slots"], top_k=case["top_k"],
                                 pow2=case["pow2"])
        return _values(s["q"], s["scales"])
    if op == "tiles":
        binding.gmm_quantize_fp8_tiles(h, s["q"], s["scales"], s["w"], pow2=case["pow2"])
        return _values(s["q"], s["scales"])
    if op == "cols":
        binding.gmm_quantize_fp8_cols(h, s["q_t"], s["t_scales"], s["x"], s["a_offsets"], row_slots=s["row_slots"],
                                      top_k=case["top_k"], q=s["q"], scales=s["scales"])
        return _values(s["q"], s["scales"], s["q_t"], s["t_scales"])
    binding.gmm_weight_grad_fp8(h, s["d_b"], s["d_t"], s["d_t_scales"], s["a_t"], s["a_t_scales"], s["a_offsets"])
    return {"d_b": s["d_b"]}


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits

def _exact_route(s):
    """The choice by hand in numpy, one token's experts in the order of their keys."""
    case = s["case"]
    x = s["logits"].double().cpu().numpy()
    t, e = x.shape
    if case["scoring"] == "sigmoid":
        score = np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
    else:
        score = np.exp(x - np.log(np.exp(x).sum(1))[:, None])
    key = score if s["bias"] is None else score + s["bias"].double().cpu().numpy()
    allowed = np.ones((t, e), bool)
    if case["groups"] > 1:
        per = e // case["groups"]
        parts = np.sort(key.reshape(t, case["groups"], per), axis=2)
        total = parts[:, :, -1] + (parts[:, :, -2] if case["group_top"] == 2 else 0)
        rank = np.argsort(np.argsort(-total, axis=1, kind="stable"), axis=1, kind="stable")
        allowed = np.repeat(rank < case["top_groups"], per, axis=1)
    order = x if s["bias"] is None else key
    ids = np.argsort(np.where(allowed, -order, np.inf), axis=1, kind="stable")[:, : case["top_k"]]
    w = np.take_along_axis(score, ids, 1)
    if case["renormalise"]:
        w = w / w.sum(1, keepdims=True)
    return {"slot_experts": ids.astype(np.int32), "weights": w * case["scale"]}


def _exact_route_grad(s):
    """The gradient by automatic differentiation of the weights' definition."""
    case = s["case"]
    x = s["logits"].double().requires_grad_()
    score = torch.sigmoid(x) if case["scoring"] == "sigmoid" else torch.softmax(x, 1)
    w = score.gather(1, s["slot_experts"].long())
    if case["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    (case["scale"] * w * s["d_weights"].double()).sum().backward()
    return {"d_logits": x.grad}


def _nearest_e4m3(y):
    """|y| <= 448 in 64 bits to the nearest e4m3 value, ties to even: 3 mantissa bits, the smallest step 2^-9."""
    step = torch.ldexp(torch.ones_like(y), torch.frexp(y.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return (torch.round(y / step) * step).clamp(-TOP, TOP)


def _exact_scale(amax, pow2):
    s = amax / TOP
    m, ex = torch.frexp(s)       # s = m 2^ex, m in [0.5, 1): a power of two itself where m = 0.5
    return torch.exp2(torch.where(m == 0.5, ex - 1, ex).clamp(min=-127).double()) if pow2 else s


def _exact_block(x, pow2):
    """(values, scale) of one block of any shape per leading index: x [blocks, elements] in 64 bits."""
    amax = x.abs().amax(1)
    scale = torch.where(amax == 0, 0.0, _exact_scale(torch.where(amax == 0, 1.0, amax), pow2))
    y = x / torch.where(scale == 0, 1.0, scale)[:, None]
    return _nearest_e4m3(y), scale


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "route_grad":
        return _exact_route_grad(s)
    if op == "tiles":
        e, n, k = case["experts"], case["n"], case["k"]
        q = torch.zeros((e, n, k), dtype=torch.float64, device=DEV)
        scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device=DEV)
        nb, kb = scales.shape[1:]
        for i in range(e):
            x = torch.nn.functional.pad(s["w"][i].double(), (0, kb * BLOCK - k, 0, nb * BLOCK - n))
            x = x.unflatten(0, (nb, BLOCK)).unflatten(2, (kb, BLOCK)).permute(0, 2, 1, 3).reshape(nb * kb, -1)
            v, sc = _exact_block(x, case["pow2"])
            v = v.reshape(nb, kb, BLOCK, BLOCK).permute(0, 2, 1, 3).reshape(nb * BLOCK, kb * BLOCK)
            q[i], scales[i] = v[:n, :k], sc.reshape(nb, kb)
        return {"q": q, "scales": scales}
    off = s["a_offsets"].tolist()
    if op == "weight_grad":
        out = torch.zeros(s["d_b"].shape, dtype=torch.float64, device=DEV)
        for i in range(case["experts"]):
            first, last = off[i], off[i + 1]
            for b in range(-(-(last - first) // BLOCK)):     # block by block, the scales on the factors
                at = first // BLOCK + i + b
                cut = slice(at * BLOCK, at * BLOCK + min(BLOCK, last - first - b * BLOCK))
                parts = [s[n][:, cut].view(torch.float8_e4m3fn).double()
                         * torch.exp2(s[n + "_scales"][at].double() - 127)[:, None] for n in ("d_t", "a_t")]
                out[i].addmm_(parts[0], parts[1].t())
        return {"d_b": out}
    x = s["x"].double()
    if s["row_slots"] is not None:
        x = x[torch.div(s["row_slots"], case["top_k"], rounding_mode="floor").long()]
    r, w = x.shape
    out = {}
    if s["q"] is not None:
        nb = -(-w // BLOCK)
        v, sc = _exact_block(torch.nn.functional.pad(x, (0, nb * BLOCK - w)).reshape(r * nb, BLOCK), case.get("pow2", False))
        out.update(q=v.reshape(r, nb * BLOCK)[:, :w], scales=sc.reshape(r, nb))
    if op == "cols":
        out["q_t"] = torch.zeros(s["q_t"].shape, dtype=torch.float64, device=DEV)
        out["t_scales"] = torch.full(s["t_scales"].shape, 2.0 ** -127, dtype=torch.float64, device=DEV)
        for i in range(case["experts"]):
            for b, first in enumerate(range(off[i], off[i + 1], BLOCK)):
                at = off[i] // BLOCK + i + b
                part = x[first:min(first + BLOCK, off[i + 1])].t()
                v, sc = _exact_block(part, True)
                out["q_t"][:, at * BLOCK:at * BLOCK + part.shape[1]] = v
                out["t_scales"][at] = torch.where(sc == 0, 2.0 ** -127, sc)
    return out
