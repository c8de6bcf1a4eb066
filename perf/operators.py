"""Cases for the operators around the grouped GEMM: tokens sorted by expert and
back (with the gradient), 4-bit floating point quantisation, and the 4-bit grouped
product.

`run` computes a case either in its plain form (elementary torch operations in 32
bits) or, where `own` is true, through the library's entry points.  Sizes are those
of the library's named workloads (decode, prefill, fine_grained) or generic.
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"nvfp4": 16, "mxfp4": 32}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ITEM = {"bf16": 2, "fp16": 2, "fp32": 4}
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # A decode step's 256 tokens to their 8 of 64 experts: latency counts.
        dict(name="dispatch_decode", op="dispatch", tokens=256, top_k=8, experts=64, width=2048, dtype="bf16",
             skew=1.1, drop=0.0),
        # A prefill batch, top-2 over 8 experts: one pass over 400 MB.
        dict(name="dispatch_prefill", op="dispatch", tokens=16384, top_k=2, experts=8, width=4096, dtype="bf16",
             skew=0.0, drop=0.0),
        # One token's 8 expert rows back into its output: the smallest call of a serving loop.
        dict(name="combine_one", op="combine", tokens=1, top_k=8, experts=64, width=2048, dtype="bf16", skew=1.1,
             drop=0.0, weights=True),
        # The fine-grained layer's 32768 rows back to 4096 tokens.
        dict(name="combine_fine", op="combine", tokens=4096, top_k=8, experts=128, width=4096, dtype="bf16",
             skew=1.0, drop=0.0, weights=True),
        # Training, prefill shapes: the gradients of the weighted sum.
        dict(name="combine_grad_prefill", op="combine_grad", tokens=16384, top_k=2, experts=8, width=4096,
             dtype="bf16", skew=0.0, drop=0.0, weights=True),
        # A small fp32 training step with an odd token count, odd width and slots over capacity dropped.
        dict(name="combine_grad_odd", op="combine_grad", tokens=1003, top_k=6, experts=64, width=1411,
             dtype="fp32", skew=1.1, drop=0.1, weights=True),
        # A decode step's activations quantised while they are gathered by expert.
        dict(name="quantize_decode", op="quantize", rows=2048, tokens=256, top_k=8, width=2048, dtype="bf16",
             fmt="nvfp4"),
        # A prefill batch's sorted rows quantised.
        dict(name="quantize_prefill", op="quantize", rows=32768, tokens=0, top_k=1, width=4096, dtype="bf16",
             fmt="mxfp4"),
        # One token's 8 experts of 64: the smallest product, bound by its weights' way to the SMs.
        dict(name="product_one", op="product", rows=8, experts=64, n=2816, k=2048, fmt="nvfp4", skew=-1.0, skip=0),
        # A decode step's 2048 rows over 64 experts: bound by the weights' bytes.
        dict(name="product_decode", op="product", rows=2048, experts=64, n=2816, k=2048, fmt="nvfp4", skew=1.1,
             skip=0),
        # A prefill batch: bound by the tensor cores.
        dict(name="product_prefill", op="product", rows=32768, experts=8, n=14336, k=4096, fmt="nvfp4", skew=0.0,
             skip=0),
        # Many experts of uneven load, some groups skipped.
        dict(name="product_fine", op="product", rows=32768, experts=128, n=4096, k=7168, fmt="mxfp4", skew=1.0,
             skip=13),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, lo, hi, steps=(1,)):
    """An odd multiple of one of `steps`, spread over the logarithm of lo .. hi: sizes that only just meet an
    alignment are as frequent as rounder ones."""
    step = rng.choice([s for s in steps if s <= hi])
    return step * (max(lo // step, min((hi // step - 1), _log(rng, max(1.0, lo / step), hi / step))) | 1)


def draw(rng):
    op = rng.choice(("dispatch", "combine", "combine_grad", "quantize", "product"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op == "quantize":
        fmt = rng.choice(("nvfp4", "mxfp4"))
        width = _odd(rng, 64, 8192, (32, 64, 256))
        rows = _odd(rng, 1, min(32768, 128 * 1024 * 1024 // width))
        top_k = rng.choice((0, 0, 1, 2, 8))
        tokens = 0
        if top_k:
            tokens = max(1, rows // top_k) | 1
            rows = tokens * top_k
        return dict(op=op, rows=rows, tokens=tokens, top_k=max(1, top_k), width=width, dtype=dtype, fmt=fmt)
    if op == "product":
        n, k = _odd(rng, 128, 14336, (8, 64, 256)), _odd(rng, 128, 7168, (32, 64, 256))
        experts = max(1, min(_log(rng, 1, 128), 3_700_000_000 // (n * k)))
        rows = _odd(rng, 1, max(2, min(32768, int(1.6e12 / (n * k)))))
        return dict(op=op, rows=rows, experts=experts, n=n, k=k, fmt=rng.choice(("nvfp4", "mxfp4")),
                    skew=rng.choice((0.0, 1.0, 1.1)), skip=rng.choice((0, experts // 8)))
    width = _odd(rng, 64, 8192, (1, 8, 64))
    experts = _log(rng, 2, 256)
    top_k = min(experts, rng.choice((1, 2, 4, 6, 8)))
    tokens = _odd(rng, 1, max(2, min(16384, 64 * 1024 * 1024 // (width * top_k))))
    case = dict(op=op, tokens=tokens, top_k=top_k, experts=experts, width=width, dtype=dtype,
                skew=rng.choice((0.0, 1.0, 1.1)), drop=rng.choice((0.0, 0.0, 0.1)))
    if op != "dispatch":
        case["weights"] = op == "combine_grad" or rng.random() < 0.7
    return case


def work(case):
    op = case["op"]
    if op in ("dispatch", "combine", "combine_grad"):
        t, s = case["tokens"], case["tokens"] * case["top_k"]
        es, d, used = ITEM[case["dtype"]], case["width"], 1.0 - case["drop"]
        if op == "dispatch":
            return {"bytes": 4 * s + t * d * es + used * s * d * es + 8 * s + 4 * (case["experts"] + 1), "flops": 0}
        if op == "combine":
            return {"bytes": used * s * d * es + t * d * es + 8 * s, "flops": 2.0 * used * s * d}
        return {"bytes": t * d * es + 2 * used * s * d * es + 12 * s, "flops": 3.0 * used * s * d}
    b = BLOCK[case["fmt"]]
    if op == "quantize":
        r, k, es = case["rows"], case["width"], ITEM[case["dtype"]]
        coded = r * k * (0.5 + 1.0 / b)
        return {"bytes": (case["tokens"] or r) * k * es + 2 * coded + r * k * 2 + (4 * r if case["tokens"] else 0),
                "flops": 2.0 * r * k}
    loads, ids = _loads(case, 0)
    rows = sum(x for x, e in zip(loads, ids) if e >= 0)
    active = sum(1 for x, e in zip(loads, ids) if e >= 0 and x > 0)
    n, k = case["n"], case["k"]
    return {"bytes": (active * n + rows) * k * (0.5 + 1.0 / b) + rows * n * 2.0, "flops": 2.0 * rows * n * k}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 11)
    return g


def _choose_experts(case, g):
    """int32 [tokens, top_k]: each token's experts, all different, expert e drawn with
    weight (e + 1)^-skew (the largest of log weight plus Gumbel noise); a share `drop`
    of the slots is -1."""
    t, e = case["tokens"], case["experts"]
    u = torch.rand((t, e), generator=g, device=DEV).clamp_(1e-9, 1 - 1e-7)
    score = -torch.log(-torch.log(u)) - case["skew"] * torch.log(torch.arange(1, e + 1, device=DEV, dtype=torch.float32))
    ids = score.topk(case["top_k"], dim=1).indices.to(torch.int32)
    gone = torch.rand(ids.shape, generator=g, device=DEV) < case["drop"]
    return torch.where(gone, torch.full_like(ids, -1), ids).contiguous()


def _randn(shape, g, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(DTYPES[dtype])


def _loads(case, seed):
    """Rows of each group, and its expert id (-1: skipped)."""
    rng = np.random.default_rng([int(seed), 5])
    e = case["experts"]
    if case["skew"] < 0:      # rows spread over as many experts, one each
        loads = np.zeros(e, np.int64)
        loads[rng.permutation(e)[: case["rows"]]] = 1
        loads[0] += case["rows"] - loads.sum()
    else:
        p = np.arange(1, e + 1, dtype=np.float64) ** -case["skew"]
        loads = rng.multinomial(case["rows"], p / p.sum())
    ids = np.arange(e, dtype=np.int32)
    ids[rng.permutation(e)[: case["skip"]]] = -1
    return [int(x) for x in loads], [int(x) for x in ids]


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("dispatch", "combine", "combine_grad"):
        t, k, d, e = case["tokens"], case["top_k"], case["width"], case["experts"]
        slot_experts = _choose_experts(case, g)
        if op == "dispatch":
            s["slot_experts"] = slot_experts
            s["tokens"] = _randn((t, d), g, case["dtype"])
            s["a_offsets"] = torch.zeros(e + 1, dtype=torch.int32, device=DEV)
            s["slot_rows"] = torch.zeros((t, k), dtype=torch.int32, device=DEV)
            s["row_slots"] = torch.zeros(t * k, dtype=torch.int32, device=DEV)
            s["rows"] = torch.zeros((t * k, d), dtype=DTYPES[case["dtype"]], device=DEV)
            return s
        s["slot_rows"] = _sort(slot_experts, e)[1]
        s["rows"] = _randn((t * k, d), g, case["dtype"])
        w = torch.rand((t, k), generator=g, device=DEV) + 0.05
        s["weights"] = w / w.sum(1, keepdim=True) if case["weights"] else None
        if op == "combine":
            s["out"] = torch.zeros((t, d), dtype=DTYPES[case["dtype"]], device=DEV)
        else:
            s["d_out"] = _randn((t, d), g, case["dtype"])
            s["d_rows"] = torch.zeros((t * k, d), dtype=DTYPES[case["dtype"]], device=DEV)
            s["d_weights"] = torch.zeros((t, k), device=DEV)
        return s
    fmt, b = case["fmt"], BLOCK[case["fmt"]]
    if op == "quantize":
        r, k = case["rows"], case["width"]
        x = torch.randn((case["tokens"] or r, k), generator=g, device=DEV)
        # A few channels an order of magnitude above the rest, as activations have them.
        x *= torch.where(torch.rand(k, generator=g, device=DEV) < 0.02, 12.0, 1.0)
        s["x"] = x.to(DTYPES[case["dtype"]])
        s["row_slots"] = None
        if case["tokens"]:
            s["row_slots"] = torch.randperm(r, generator=g, device=DEV).to(torch.int32)
        s["global"] = (s["x"].float().abs().amax() / (6 * 448)).reshape(1) if fmt == "nvfp4" else None
        s["packed"] = torch.zeros((r, k // 2), dtype=torch.uint8, device=DEV)
        s["scales"] = torch.zeros((r, _pitch(k, b)), dtype=torch.uint8, device=DEV)
        s["values"] = torch.zeros((r, k), dtype=torch.bfloat16, device=DEV)
        return s
    n, k, e = case["n"], case["k"], case["experts"]
    s["loads"], s["ids"] = _loads(case, seed)
    r = sum(s["loads"])
    s["a_offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(s["loads"])]), dtype=torch.int32, device=DEV)
    s["expert_ids"] = torch.tensor(s["ids"], dtype=torch.int32, device=DEV)
    s["a_global"] = torch.full((1,), 4.5 / (6 * 448), device=DEV) if fmt == "nvfp4" else None
    s["b_global"] = torch.empty(e, device=DEV) if fmt == "nvfp4" else None
    s["a"], s["a_scales"] = _encode(torch.randn((r, k), generator=g, device=DEV), fmt, s["a_global"])
    s["b"] = torch.empty((e, n, k // 2), dtype=torch.uint8, device=DEV)
    s["b_scales"] = torch.empty((e, n, _pitch(k, b)), dtype=torch.uint8, device=DEV)
    for i in range(e):
        w = torch.randn((n, k), generator=g, device=DEV) * 0.02
        if fmt == "nvfp4":
            s["b_global"][i] = w.abs().amax() / (6 * 448)
        s["b"][i], s["b_scales"][i] = _encode(w, fmt, s["b_global"][i] if fmt == "nvfp4" else None)
    s["c"] = torch.zeros((r, n), dtype=torch.bfloat16, device=DEV)
    s["stats"] = torch.zeros(2, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

def _sort(slot_experts, experts):
    """(a_offsets, slot_rows, row_slots) of the stable order by expert."""
    e = slot_experts.reshape(-1)
    slots = torch.arange(e.numel(), device=DEV, dtype=torch.int32)
    one_hot = (e[:, None] == torch.arange(experts, device=DEV, dtype=torch.int32)).to(torch.int32)
    seen = torch.cumsum(one_hot, 0, dtype=torch.int32)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(seen[-1], 0, dtype=torch.int32)
    valid = (e >= 0) & (e < experts)
    own_e = e.clamp(0, experts - 1).long()
    row = offsets[own_e] + seen.gather(1, own_e[:, None])[:, 0] - 1
    slot_rows = torch.where(valid, row, -1)
    row_slots = torch.full((e.numel() + 1,), -1, dtype=torch.int32, device=DEV)
    row_slots[torch.where(valid, row, e.numel()).long()] = slots
    return offsets, slot_rows.reshape(slot_experts.shape), row_slots[:-1]


def _pitch(k, block):
    """Bytes of a row of block scales: padded to 16."""
    return -(-(k // block) // 16) * 16


def _power_of_two(code):
    """The value of an e8m0 code: 2^(code - 127)."""
    code = code.to(torch.int32)
    return torch.where(code == 0, 0x00400000, code << 23).view(torch.float32)


def _quantize(x, fmt, global_scale):
    """x [rows, k] in fp32 -> signed e2m1 magnitude codes, scale bytes and the value a scale stands for."""
    b = BLOCK[fmt]
    blocks = x.reshape(x.shape[0], -1, b)
    amax = blocks.abs().amax(2)
    if fmt == "nvfp4":
        g = 1.0 if global_scale is None else global_scale.reshape(())
        s8 = (amax / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
        scale, codes = s8.float() * g, s8.view(torch.uint8)
    else:
        exponent = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
        codes = torch.where(amax == 0, 0, exponent + 127).to(torch.uint8)
        scale = _power_of_two(codes)
    y = blocks.abs() / torch.where(scale == 0, 1.0, scale)[:, :, None]
    y = torch.where(scale[:, :, None] == 0, 0.0, y)
    # Round to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code.
    q = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    return q.to(torch.uint8).reshape(x.shape), codes, scale


def _encode(x, fmt, global_scale):
    """Packed e2m1 pairs (even k in the low nibble) and padded scale bytes."""
    q, codes, _ = _quantize(x, fmt, global_scale)
    q = q | ((x < 0).to(torch.uint8) << 3)
    scales = torch.zeros((x.shape[0], _pitch(x.shape[1], BLOCK[fmt])), dtype=torch.uint8, device=DEV)
    scales[:, : codes.shape[1]] = codes
    return q[:, 0::2] | (q[:, 1::2] << 4), scales


def _decode(packed, scales, fmt):
    """fp32 values without the global scale."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    byte = torch.arange(256, device=DEV)
    pairs = torch.stack([lut[byte & 15], lut[byte >> 4]], 1)
    rows, k = packed.shape[0], packed.shape[1] * 2
    b = BLOCK[fmt]
    code = scales[:, : k // b]
    scale = code.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else _power_of_two(code)
    return (pairs[packed.int()].reshape(rows, k // b, b) * scale[:, :, None]).reshape(rows, k)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "dispatch":
        offsets, slot_rows, row_slots = _sort(s["slot_experts"], case["experts"])
        rows = s["tokens"][row_slots.clamp(min=0).long() // case["top_k"]]
        rows = torch.where((row_slots >= 0)[:, None], rows, s["rows"])
        return {"a_offsets": offsets, "slot_rows": slot_rows, "row_slots": row_slots, "rows": rows}
    if op in ("combine", "combine_grad"):
        valid = s["slot_rows"] >= 0
        at = s["slot_rows"].clamp(min=0).long()
        w = valid.float() if s["weights"] is None else torch.where(valid, s["weights"], 0.0)
        if op == "combine":
            return {"out": (s["rows"][at].float() * w[:, :, None]).sum(1).to(s["rows"].dtype)}
        d_out = s["d_out"].float()
        d_weights = torch.where(valid, (s["rows"][at].float() * d_out[:, None, :]).sum(2), 0.0)
        d_slots = (w[:, :, None] * d_out[:, None, :]).to(s["rows"].dtype).reshape(-1, case["width"])
        d_rows = torch.cat([s["d_rows"], s["d_rows"][:1]])
        d_rows[torch.where(valid, at, d_rows.shape[0] - 1).reshape(-1)] = d_slots
        return {"d_rows": d_rows[:-1], "d_weights": d_weights}
    fmt = case["fmt"]
    if op == "quantize":
        x = s["x"] if s["row_slots"] is None else s["x"][s["row_slots"].long() // case["top_k"]]
        x = x.float()
        q, codes, scale = _quantize(x, fmt, s["global"])
        value = torch.tensor(E2M1, device=DEV)[q.int()] * torch.where(x < 0, -1.0, 1.0)
        value = value.reshape(x.shape[0], -1, BLOCK[fmt]) * scale[:, :, None]
        out = {"values": value.reshape(x.shape).to(torch.bfloat16)}
        if fmt == "nvfp4":
            out["scales"] = codes.view(torch.float8_e4m3fn)
        return out
    a = _decode(s["a"], s["a_scales"], fmt)
    at = [sum(s["loads"][:i]) for i in range(len(s["loads"]) + 1)]
    ga = 1.0 if s["a_global"] is None else s["a_global"]

    def group(i, e):
        if e < 0:
            return s["c"][at[i]:at[i + 1]]
        gb = 1.0 if s["b_global"] is None else s["b_global"][e]
        y = a[at[i]:at[i + 1]] @ _decode(s["b"][e], s["b_scales"][e], fmt).t()
        return (y * (ga * gb)).to(torch.bfloat16)

    c = torch.cat([group(i, e) for i, e in enumerate(s["ids"]) if s["loads"][i]])
    return {"c": c, "active": (s["expert_ids"] >= 0).sum()}


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
    h = _handle(case.get("experts", 1))
    if op == "dispatch":
        binding.gmm_dispatch(h, s["a_offsets"], s["slot_rows"], s["row_slots"], s["slot_experts"], rows=s["rows"],
                             tokens=s["tokens"])
        return {k: s[k] for k in ("a_offsets", "slot_rows", "row_slots", "rows")}
    if op == "combine":
        binding.gmm_combine(h, s["out"], s["rows"], s["slot_rows"], weights=s["weights"])
        return {"out": s["out"]}
    if op == "combine_grad":
        binding.gmm_combine_grad(h, s["d_rows"], s["d_weights"], s["d_out"], s["rows"], s["slot_rows"],
                                 weights=s["weights"])
        return {"d_rows": s["d_rows"], "d_weights": s["d_weights"]}
    fmt = case["fmt"]
    if op == "quantize":
        binding.gmm_quantize_fp4(h, s["packed"], s["scales"], s["x"], fmt=fmt, row_slots=s["row_slots"],
                                 top_k=case["top_k"], global_scale=s["global"])
        binding.gmm_dequantize_fp4(h, s["values"], s["packed"], s["scales"], fmt=fmt, global_scale=s["global"])
        out = {"values": s["values"]}
        if fmt == "nvfp4":
            out["scales"] = s["scales"][:, : case["width"] // 16].view(torch.float8_e4m3fn)
        return out
    binding.gmm_run_fp4(h, s["c"], s["a"], s["a_offsets"], s["b"], s["expert_ids"], s["stats"], s["a_scales"],
                        s["b_scales"], fmt=fmt, a_global=s["a_global"], b_global=s["b_global"])
    return {"c": s["c"], "active": s["stats"][1].to(torch.int64)}


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits

def _exact_power(e):
    """2^e in 64 bits, from the exponent's bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_e2m1(y):
    """|y| in 64 bits to the nearest e2m1 value, ties to the even code, by distances."""
    values = torch.tensor(E2M1, dtype=torch.float64, device=y.device)
    best, code = (y - 0.0).abs(), torch.zeros(y.shape, dtype=torch.int64, device=y.device)
    for i in range(1, 8):
        far = (y - values[i]).abs()
        take = (far < best) | ((far == best) & (i % 2 == 0))
        best, code = torch.where(take, far, best), torch.where(take, i, code)
    return values[code]


def _exact_values(packed, scales, fmt):
    """Decoded values in 64 bits, from the formats' bit fields."""
    def e2m1(c):
        c = c.to(torch.int64)
        ex, m = (c >> 1) & 3, (c & 1).double()
        v = torch.where(ex == 0, 0.5 * m, (1.0 + 0.5 * m) * _exact_power(ex - 1))
        return torch.where((c & 8) != 0, -v, v)

    b = BLOCK[fmt]
    k = packed.shape[1] * 2
    q = torch.stack([e2m1(packed & 15), e2m1(packed >> 4)], 2).reshape(packed.shape[0], k)
    c = scales[:, : k // b].to(torch.int64)
    if fmt == "nvfp4":
        ex, m = (c >> 3) & 15, (c & 7).double()
        sv = torch.where(ex == 0, m / 512, (1.0 + m / 8) * _exact_power(ex - 7))
    else:
        sv = _exact_power(c - 127)
    return q * sv.repeat_interleave(b, 1)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "dispatch":
        e = s["slot_experts"].cpu().numpy().reshape(-1)
        order = np.argsort(np.where(e < 0, case["experts"], e), kind="stable")
        count = int((e >= 0).sum())
        slot_rows = np.full(e.size, -1, np.int32)
        slot_rows[order[:count]] = np.arange(count)
        row_slots = np.full(e.size, -1, np.int32)
        row_slots[:count] = order[:count]
        offsets = np.concatenate([[0], np.cumsum(np.bincount(e[e >= 0], minlength=case["experts"]))]).astype(np.int32)
        rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device=DEV)
        pick = torch.from_numpy(order[:count] // case["top_k"]).to(DEV)
        rows[:count] = s["tokens"].double()[pick]
        return {"a_offsets": offsets, "slot_rows": slot_rows.reshape(s["slot_rows"].shape), "row_slots": row_slots,
                "rows": rows}
    if op in ("combine", "combine_grad"):
        t, k, d = case["tokens"], case["top_k"], case["width"]
        w = torch.ones((t, k), dtype=torch.float64, device=DEV) if s["weights"] is None else s["weights"].double()
        out = torch.zeros((t, d), dtype=torch.float64, device=DEV)
        d_rows = torch.zeros((t * k, d), dtype=torch.float64, device=DEV)
        d_weights = torch.zeros((t, k), dtype=torch.float64, device=DEV)
        for j in range(k):
            has = torch.nonzero(s["slot_rows"][:, j] >= 0)[:, 0]
            at = s["slot_rows"][has, j].long()
            picked = s["rows"][at].double()
            if op == "combine":
                out[has] += w[has, j][:, None] * picked
            else:
                g = s["d_out"][has].double()
                d_rows[at] = w[has, j][:, None] * g
                d_weights[has, j] = (g * picked).sum(1)
        return {"out": out} if op == "combine" else {"d_rows": d_rows, "d_weights": d_weights}
    fmt = case["fmt"]
    if op == "quantize":
        x = s["x"] if s["row_slots"] is None else s["x"][torch.div(s["row_slots"], case["top_k"], rounding_mode="floor").long()]
        b = BLOCK[fmt]
        blocks = x.double().reshape(x.shape[0], -1, b)
        amax = blocks.abs().amax(2)
        if fmt == "nvfp4":
            g = s["global"].double()
            t = amax / (6 * g)
            # e4m3: 3 mantissa bits, the smallest step 2^-9, the largest value 448.
            step = _exact_power(torch.frexp(t.clamp(min=2.0 ** -6)).exponent - 4)
            s8 = torch.round(t / step) * step
            s8 = s8.clamp(max=448.0)
            scale = s8 * g
        else:
            scale = _exact_power(torch.frexp(amax.clamp(min=2.0 ** -125)).exponent - 3)
        y = torch.where(scale[:, :, None] == 0, 0.0, blocks.abs() / torch.where(scale == 0, 1.0, scale)[:, :, None])
        v = _exact_e2m1(y) * torch.sign(blocks) * scale[:, :, None]
        out = {"values": v.reshape(x.shape)}
        if fmt == "nvfp4":
            out["scales"] = s8
        return out
    a = _exact_values(s["a"], s["a_scales"], fmt)
    if s["a_global"] is not None:
        a = a * s["a_global"].double()
    c = torch.zeros((a.shape[0], case["n"]), dtype=torch.float64, device=DEV)
    r = 0
    for load, e in zip(s["loads"], s["ids"]):
        if load and e >= 0:
            w = _exact_values(s["b"][e], s["b_scales"][e], fmt)
            if s["b_global"] is not None:
                w = w * s["b_global"][e].double()
            c[r:r + load] = a[r:r + load] @ w.t()
        r += load
    return {"c": c, "active": sum(1 for e in s["ids"] if e >= 0)}
