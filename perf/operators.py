"""The routed-expert operators: cases over their real range, and the same operators in plain torch.

``run`` computes a case with elementary torch operations in 32 bits where ``own`` is
false, and with the package's calls where it is true. ``exact`` is the definition in 64
bits. Sizes are those of the package's synthetic workloads (hidden 7168 and 1024, 256
experts of which a token takes 8, projections 7168 -> 1536 and 16384 -> 7168) with an
expert width of 2048, and tokens from one to a prompt's.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
BLOCK = 128            # values that share a scale
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100   # a block's largest magnitude counts as at least this


# ----------------------------------------------------------------- cases

def listed():
    return [
        # a decode batch of the router's benchmark: every expert on this GPU, weights normalised
        {"name": "sort_decode", "op": "sort", "tokens": 128, "k": 8, "experts": 256, "first": 0, "local": 256,
         "normalize": True},
        # a prompt chunk of odd length on one of eight expert-parallel ranks: most choices are elsewhere
        {"name": "sort_prompt_shard", "op": "sort", "tokens": 12289, "k": 8, "experts": 256, "first": 64, "local": 32,
         "normalize": True},
        # one decode token, its row quantised for the 8-bit product
        {"name": "gather_one", "op": "gather", "tokens": 1, "hidden": 7168, "k": 8, "experts": 256, "first": 0,
         "local": 256, "dtype": "bf16", "fp8": True},
        # a prompt chunk, quantised on the way
        {"name": "gather_prompt", "op": "gather", "tokens": 4096, "hidden": 7168, "k": 8, "experts": 256, "first": 0,
         "local": 256, "dtype": "bf16", "fp8": True},
        # the way back of that chunk, weights applied
        {"name": "combine_prompt", "op": "combine", "tokens": 4096, "hidden": 7168, "k": 8, "experts": 256, "first": 0,
         "local": 256, "dtype": "bf16", "weighted": True, "backward": False},
        # its gradient, at an odd token count
        {"name": "combine_backward", "op": "combine", "tokens": 2999, "hidden": 7168, "k": 8, "experts": 256,
         "first": 0, "local": 256, "dtype": "bf16", "weighted": True, "backward": True},
        # gate and up projections of a decode batch's rows -> activated, quantised
        {"name": "gated_decode", "op": "quantize", "rows": 1024, "cols": 2048, "dtype": "bf16", "gated": True},
        # of a prompt chunk's rows
        {"name": "gated_prompt", "op": "quantize", "rows": 32768, "cols": 2048, "dtype": "bf16", "gated": True},
        # one token through the query down-projection
        {"name": "matmul_one", "op": "matmul", "rows": 1, "features": 1536, "inner": 7168, "dtype": "bf16"},
        # a prompt chunk through the output projection
        {"name": "matmul_prompt", "op": "matmul", "rows": 4096, "features": 7168, "inner": 16384, "dtype": "bf16"},
        # the gate and up product of a decode batch of 128 tokens on one of eight expert-parallel ranks
        {"name": "grouped_decode", "op": "grouped", "tokens": 128, "k": 8, "experts": 256, "first": 32, "local": 32,
         "features": 4096, "inner": 7168, "dtype": "bf16"},
        # of a prompt chunk of odd length
        {"name": "grouped_prompt", "op": "grouped", "tokens": 8191, "k": 8, "experts": 256, "first": 32, "local": 32,
         "features": 4096, "inner": 7168, "dtype": "bf16"},
    ]


def _log_int(rng, low, high, step=1):
    v = math.exp(rng.uniform(math.log(low), math.log(high + 1)))
    return min(high, max(low, int(v) // step * step))


def draw(rng):
    op = rng.choice(["sort", "gather", "combine", "quantize", "matmul", "grouped"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    experts = rng.choice([64, 80, 96, 128, 256, 512])
    shards = rng.choice([1, 1, 2, 8])
    local = experts // shards
    place = {"k": rng.randint(1, 10), "experts": experts, "first": local * rng.randrange(shards), "local": local}
    fewest = 1 if shards == 1 else 64     # a shard of a few tokens' choices would often have none
    if op == "sort":
        return {"op": op, "tokens": _log_int(rng, fewest, 16384), **place, "normalize": rng.random() < 0.5}
    if op == "gather":
        return {"op": op, "tokens": _log_int(rng, fewest, 3000), "hidden": _log_int(rng, 256, 7168, 16), **place,
                "dtype": dtype, "fp8": rng.random() < 0.5}
    if op == "combine":
        return {"op": op, "tokens": _log_int(rng, fewest, 2000), "hidden": _log_int(rng, 256, 7168, 16), **place,
                "dtype": dtype, "weighted": rng.random() < 0.7, "backward": rng.random() < 0.5}
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "cols": _log_int(rng, 256, 4096, 16), "dtype": dtype,
                "gated": rng.random() < 0.6}
    if op == "matmul":
        return {"op": op, "rows": _log_int(rng, 1, 4096), "features": _log_int(rng, 256, 7168, 16),
                "inner": _log_int(rng, 256, 16384, 16), "dtype": dtype}
    shard = rng.random() < 0.5            # else every expert is here
    held = rng.choice([16, 24, 32])
    place.update(experts=held * 4 if shard else held, local=held, first=held if shard else 0)
    n, inner = _log_int(rng, 256, 4096, 16), _log_int(rng, 256, 7168, 16)
    most = int(9e11 / (2 * n * inner * place["k"] * held / place["experts"]))
    return {"op": op, "tokens": _log_int(rng, 64 if shard else 1, min(8191, most)), **place, "features": n,
            "inner": inner, "dtype": dtype}


# ----------------------------------------------------------------- inputs

def _route(case, g):
    """Top-K choices of a router whose experts differ in how often they are taken, and its affinities."""
    t, k, e = case["tokens"], case["k"], case["experts"]
    logits = torch.randn(t, e, generator=g, device=DEVICE) + 0.5 * torch.randn(e, generator=g, device=DEVICE)
    top, idx = torch.topk(logits, k, dim=1)
    aff = torch.zeros(t, e, device=DEVICE).scatter_(1, idx, torch.sigmoid(top)).to(torch.bfloat16)
    return idx.to(torch.int32), aff


def _sorted_rows(case, idx):
    """(offsets, row_of, source_of) of the assignments in expert order."""
    n = case["tokens"] * case["k"]
    e = idx.reshape(-1).long() - case["first"]
    here = (e >= 0) & (e < case["local"])
    key = torch.where(here, e, case["local"])
    order = torch.sort(key, stable=True).indices
    at = torch.empty_like(order)
    at[order] = torch.arange(n, device=DEVICE)
    counts = torch.zeros(case["local"] + 1, dtype=torch.long, device=DEVICE).index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([counts.new_zeros(1), counts[:-1].cumsum(0)])
    row_of = torch.where(here, at, -1).reshape(idx.shape)
    source_of = torch.where(torch.arange(n, device=DEVICE) < offsets[-1], order, -1)
    return offsets.to(torch.int32), row_of.to(torch.int32), source_of.to(torch.int32)


def _hidden(rows, cols, dtype, g):
    """Activations: normal values, a few channels of them much larger, as hidden states have them."""
    big = torch.where(torch.rand(cols, generator=g, device=DEVICE) < 0.01, 8.0, 1.0)
    return (torch.randn(rows, cols, generator=g, device=DEVICE) * big).to(dtype)


def _weight(experts, n, k, g):
    """Weights of N(0, 1 / k) as e4m3 with a scale for each 128 x 128 block."""
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    w = torch.stack([(torch.randn(n, k, generator=g, device=DEVICE) * 100).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
                     .view(torch.uint8) for _ in range(experts)]).view(E4M3)
    s = torch.exp(0.3 * torch.randn(experts, nb, kb, generator=g, device=DEVICE)) / (100 * math.sqrt(k))
    return w, s


def _buffer(*shape, dtype):
    return torch.zeros(shape, dtype=torch.uint8 if dtype == E4M3 else dtype, device=DEVICE).view(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s, op = {"case": case}, case["op"]
    dtype = DTYPES.get(case.get("dtype"))
    if op in ("sort", "gather", "combine", "grouped"):
        t, k = case["tokens"], case["k"]
        idx, aff = _route(case, g)
        r = t * k
    if op in ("gather", "combine", "grouped"):
        s["offsets"], s["row_of"], _ = _sorted_rows(case, idx)
    if op == "sort":
        s.update(idx=idx, aff=aff, scale=2.5, offsets=_buffer(case["local"] + 1, dtype=torch.int32),
                 row_of=_buffer(t, k, dtype=torch.int32), source_of=_buffer(r, dtype=torch.int32),
                 weights=_buffer(t, k, dtype=torch.float32),
                 workspace=torch.empty((r // 1024 + 2) * case["local"] * 4 + 4096, dtype=torch.uint8, device=DEVICE))
    elif op == "gather":
        h = case["hidden"]
        s["x"] = _hidden(t, h, dtype, g)
        s["rows"] = _buffer(r, h, dtype=E4M3 if case["fp8"] else dtype)
        s["scales"] = _buffer(-(-h // BLOCK), r, dtype=torch.float32) if case["fp8"] else None
    elif op == "combine":
        h = case["hidden"]
        s["rows"] = _hidden(r, h, dtype, g)
        s["weights"] = torch.rand(t, k, generator=g, device=DEVICE) if case["weighted"] else None
        if case["backward"]:
            s["grad_out"] = torch.randn(t, h, generator=g, device=DEVICE).to(dtype)
            s["grad_rows"] = _buffer(r, h, dtype=dtype)
            s["grad_weights"] = _buffer(t, k, dtype=torch.float32)
            if s["weights"] is None:   # the gradient of an unweighted sum: weights of one
                s["weights"] = torch.ones(t, k, device=DEVICE)
        else:
            s["out"] = _buffer(t, h, dtype=dtype)
    elif op == "quantize":
        r, c = case["rows"], case["cols"]
        s["x"] = _hidden(r, 2 * c if case["gated"] else c, dtype, g)
        s["q"] = _buffer(r, c, dtype=E4M3)
        s["scales"] = _buffer(-(-c // BLOCK), r, dtype=torch.float32)
    else:
        n, k = case["features"], case["inner"]
        m = case["rows"] if op == "matmul" else r
        experts = 1 if op == "matmul" else case["local"]
        s["x"], s["x_scales"] = _quantized(_hidden(m, k, torch.float32, g))
        s["w"], s["w_scales"] = _weight(experts, n, k, g)
        if op == "matmul":
            s["w"], s["w_scales"] = s["w"][0], s["w_scales"][0]
        else:
            s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())   # the longest group, for the plain form
        s["out"] = _buffer(m, n, dtype=dtype)
    return s


# ----------------------------------------------------------------- the operators, plainly

def _quantized(x):
    """Rows of fp32 as e4m3 and a scale for each 128 of a row, scales [blocks, rows]."""
    r, c = x.shape
    nb = -(-c // BLOCK)
    p = torch.nn.functional.pad(x, (0, nb * BLOCK - c)).reshape(r, nb, BLOCK)
    amax = p.abs().amax(2).clamp(min=AMAX_FLOOR)
    q = (p * (E4M3_MAX / amax)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
    return q.reshape(r, nb * BLOCK)[:, :c].contiguous(), (amax / E4M3_MAX).t().contiguous()


def _values(q, scales):
    """fp32 values of e4m3 rows with scales [blocks, rows]."""
    return q.float() * scales.t().repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _weight_values(w, scales):
    s = scales.repeat_interleave(BLOCK, -2)[..., :w.shape[-2], :].repeat_interleave(BLOCK, -1)[..., :w.shape[-1]]
    return w.float() * s


def _plain(s):
    case = s["case"]
    op, dtype = case["op"], DTYPES.get(case.get("dtype"))
    if op == "sort":
        idx = s["idx"].long()
        a = s["aff"].float().gather(1, idx)
        w = a / a.sum(1, keepdim=True) if case["normalize"] else a
        return (*_sorted_rows(case, s["idx"]), s["scale"] * w)
    if op == "quantize":
        x, c = s["x"].float(), case["cols"]
        if case["gated"]:
            x = x[:, :c] / (1 + torch.exp(-x[:, :c])) * x[:, c:]
        return _quantized(x)
    if op == "matmul":
        return (_values(s["x"], s["x_scales"]) @ _weight_values(s["w"], s["w_scales"]).t()).to(dtype)
    if op == "grouped":
        r, most = s["x"].shape[0], max(1, s["most"])
        row = torch.arange(most, device=DEVICE) + s["offsets"][:-1, None]           # [experts, most]
        inside = row < s["offsets"][1:, None]
        x = _values(s["x"], s["x_scales"])[row.clamp(max=r - 1)]
        y = torch.bmm(x, _weight_values(s["w"], s["w_scales"]).transpose(1, 2)).to(dtype)
        out = torch.zeros(r + 1, y.shape[2], dtype=dtype, device=DEVICE)            # the last row takes what is no row's
        out[torch.where(inside, row, r)] = y
        return out[:r]
    t, k = s["row_of"].shape
    row, r = s["row_of"].long(), t * k
    here = row >= 0
    if op == "gather":
        to = torch.where(here, row, r)
        out = torch.zeros(r + 1, case["hidden"], dtype=s["rows"].dtype if not case["fp8"] else torch.float32,
                          device=DEVICE)
        if not case["fp8"]:
            out[to] = s["x"][:, None]
            return out[:r]
        q, scale = _quantized(s["x"].float())
        scales = torch.zeros(r + 1, scale.shape[0], device=DEVICE)
        out[to] = q.float()[:, None]
        scales[to] = scale.t()[:, None]
        return out[:r].to(E4M3), scales[:r].t().contiguous()
    rows = torch.where(here[:, :, None], s["rows"][row.clamp(min=0)].float(), 0.0)   # [tokens, k, hidden]
    if not case["backward"]:
        return (rows if s["weights"] is None else rows * s["weights"][:, :, None]).sum(1).to(dtype)
    dout = s["grad_out"].float()[:, None]
    grad = torch.zeros(r + 1, case["hidden"], dtype=dtype, device=DEVICE)
    grad[torch.where(here, row, r)] = (dout * s["weights"][:, :, None]).to(dtype)
    return grad[:r], (dout * rows).sum(2)


def run(state):
    if not own:
        return _plain(state)
    from sparse_mla_decode_front_b200 import experts as X
    s, case = state, state["case"]
    op = case["op"]
    if op == "sort":
        X.mla_moe_sort(s["idx"], s["offsets"], s["row_of"], s["source_of"], s["workspace"], case["first"], s["aff"],
                       s["weights"], case["normalize"], s["scale"])
        return s["offsets"], s["row_of"], s["source_of"], s["weights"]
    if op == "gather":
        X.mla_moe_gather(s["x"], s["row_of"], s["rows"], s["scales"])
        return (s["rows"], s["scales"]) if case["fp8"] else s["rows"]
    if op == "combine" and not case["backward"]:
        X.mla_moe_combine(s["rows"], s["row_of"], s["weights"], s["out"])
        return s["out"]
    if op == "combine":
        X.mla_moe_combine_backward(s["grad_out"], s["rows"], s["row_of"], s["weights"], s["grad_rows"],
                                   s["grad_weights"])
        return s["grad_rows"], s["grad_weights"]
    if op == "quantize":
        X.mla_fp8_quantize(s["x"], s["q"], s["scales"], case["gated"])
        return s["q"], s["scales"]
    if op == "matmul":
        X.mla_fp8_matmul(s["x"], s["x_scales"], s["w"], s["w_scales"], s["out"])
    else:
        X.mla_fp8_grouped_matmul(s["x"], s["x_scales"], s["w"], s["w_scales"], s["offsets"], s["out"])
    return s["out"]


# ----------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}.get(case.get("dtype"), 0)
    blocks = lambda c: -(-c // BLOCK)  # noqa: E731
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        return {"bytes": r * c * (size * (2 if case["gated"] else 1) + 1) + 4 * r * blocks(c),
                "flops": r * c * (7 if case["gated"] else 3)}
    if op == "matmul":
        m, n, k = case["rows"], case["features"], case["inner"]
        return {"bytes": m * k + n * k + 4 * blocks(k) * (m + blocks(n)) + size * m * n, "flops": 2 * m * n * k}
    t, tk = case["tokens"], case["tokens"] * case["k"]
    rows = tk * case["local"] / case["experts"]     # local rows, on average
    if op == "sort":
        return {"bytes": 4 * tk + 2 * tk + 4 * (case["local"] + 1) + 12 * tk, "flops": 2 * tk}
    if op == "grouped":
        n, k = case["features"], case["inner"]
        used = case["local"] * (1 - (1 - case["k"] / case["experts"]) ** t)   # experts that have a row, on average
        return {"bytes": rows * k + used * n * k + 4 * blocks(k) * (rows + used * blocks(n)) + size * rows * n,
                "flops": 2 * rows * n * k}
    h = case["hidden"]
    if op == "gather":
        return {"bytes": size * t * h + 4 * tk + rows * (h + 4 * blocks(h) if case["fp8"] else size * h),
                "flops": 3 * t * h if case["fp8"] else 0}
    if not case["backward"]:
        return {"bytes": size * (rows + t) * h + (8 if case["weighted"] else 4) * tk, "flops": 2 * rows * h}
    return {"bytes": size * (2 * rows + t) * h + 12 * tk, "flops": 3 * rows * h}


# ----------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f8 = torch.float64

    def quant(x):
        q, scale = torch.empty_like(x), []
        for c0 in range(0, x.shape[1], BLOCK):
            part = x[:, c0:c0 + BLOCK]
            one = torch.maximum(part.abs().max(1).values, torch.tensor(AMAX_FLOOR, dtype=f8, device=DEVICE)) / E4M3_MAX
            q[:, c0:c0 + BLOCK] = part / one[:, None]
            scale.append(one)
        return q, torch.stack(scale)

    def product(x, xs, w, ws):
        out = torch.zeros(x.shape[0], w.shape[0], dtype=f8, device=DEVICE)
        wide = ws.to(f8).repeat_interleave(BLOCK, 0)[:w.shape[0]]
        for b in range(xs.shape[0]):
            part = slice(b * BLOCK, (b + 1) * BLOCK)
            out += (x[:, part].to(f8) * xs[b].to(f8)[:, None]) @ (w[:, part].to(f8) * wide[:, b:b + 1]).t()
        return out

    if op == "sort":
        a = torch.take_along_dim(s["aff"].to(f8), s["idx"].long(), 1)
        return None, None, None, s["scale"] * (a / a.sum(1, keepdim=True) if case["normalize"] else a)
    if op == "quantize":
        x, c = s["x"].to(f8), case["cols"]
        return quant(x[:, :c] * torch.sigmoid(x[:, :c]) * x[:, c:] if case["gated"] else x)
    if op == "matmul":
        return product(s["x"], s["x_scales"], s["w"], s["w_scales"])
    if op == "grouped":
        out = torch.zeros(s["out"].shape, dtype=f8, device=DEVICE)
        ends = s["offsets"].tolist()
        for e in range(case["local"]):
            part = slice(ends[e], ends[e + 1])
            out[part] = product(s["x"][part], s["x_scales"][:, part], s["w"][e], s["w_scales"][e])
        return out
    t, k = s["row_of"].shape
    r, h = t * k, case["hidden"]
    taken = [(s["row_of"][:, j] >= 0).nonzero()[:, 0] for j in range(k)]   # tokens whose j-th choice is here
    at = [s["row_of"][taken[j], j].long() for j in range(k)]
    if op == "gather":
        x = s["x"].to(f8)
        q, scale = quant(x) if case["fp8"] else (x, None)
        rows = torch.zeros(r, h, dtype=f8, device=DEVICE)
        scales = torch.zeros(-(-h // BLOCK), r, dtype=f8, device=DEVICE)
        for j in range(k):
            rows[at[j]] = q[taken[j]]
            if case["fp8"]:
                scales[:, at[j]] = scale[:, taken[j]]
        return (rows, scales) if case["fp8"] else rows
    w = torch.ones(t, k, dtype=f8, device=DEVICE) if s["weights"] is None else s["weights"].to(f8)
    if not case["backward"]:
        out = torch.zeros(t, h, dtype=f8, device=DEVICE)
        for j in range(k):
            out[taken[j]] += w[taken[j], j, None] * s["rows"][at[j]].to(f8)
        return out
    dout = s["grad_out"].to(f8)
    grad, dw = torch.zeros(r, h, dtype=f8, device=DEVICE), torch.zeros(t, k, dtype=f8, device=DEVICE)
    for j in range(k):
        grad[at[j]] = w[taken[j], j, None] * dout[taken[j]]
        dw[taken[j], j] = torch.linalg.vecdot(dout[taken[j]], s["rows"][at[j]].to(f8))
    return grad, dw
