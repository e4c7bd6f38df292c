"""Cases of the operators that join causal layers to the stack's frames: cross attention of packed or
single rows to memories of frames, and the matrix product with bias, activation and residual.

``run`` computes a case in plain torch operations (``own`` false) or through the package's entry
points (``own`` true); ``exact`` computes it in 64 bits from the definitions.
"""

import math
import random

import torch

own = False

TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
EIGHT = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}
RUN = 64  # rows of one run of the plain attention
SLOPE = 0.01
MOST_ATTENTION = 5.5e11  # flops of the largest attention
MOST_MEMORY = 3.2e8  # elements of k and v together
MOST_PRODUCT = 4.3e11  # flops of the largest product


def listed():
    return [
        # one new row of one stream reads one window of 589 frames at the stack's output width: launch latency
        {"name": "cross_row_one", "op": "cross_step", "rows": 1, "heads": 4, "kv_heads": 4, "width": 64, "frames": 589,
         "layout": "padded", "ragged": False, "masked": False, "type": "bfloat16"},
        # one new row of each of 256 streams: the windows' bytes
        {"name": "cross_rows_many", "op": "cross_step", "rows": 256, "heads": 16, "kv_heads": 4, "width": 64, "frames": 589,
         "layout": "padded", "ragged": False, "masked": False, "type": "bfloat16"},
        # four hypotheses of each of 32 streams read long recordings of unequal lengths, silent frames left out
        {"name": "cross_hypotheses", "op": "cross", "rows": 128, "sequences": 32, "uneven": False, "heads": 32,
         "kv_heads": 8, "width": 128, "frames": 4096, "layout": "padded", "ragged": True, "masked": True, "type": "float16"},
        # 64 rows for each of 32 windows of 589 frames, 32 bits
        {"name": "cross_windows_fp32", "op": "cross", "rows": 2048, "sequences": 32, "uneven": False, "heads": 4,
         "kv_heads": 4, "width": 64, "frames": 589, "layout": "padded", "ragged": False, "masked": False, "type": "float32"},
        # one prompt alone and one long recording: few tiles, the frames have to be split
        {"name": "cross_one_prompt", "op": "cross", "rows": 500, "sequences": 1, "uneven": False, "heads": 16, "kv_heads": 16,
         "width": 64, "frames": 4096, "layout": "padded", "ragged": False, "masked": False, "type": "bfloat16"},
        # a packed batch of prompts and of recordings, all of unequal lengths
        {"name": "cross_prompts", "op": "cross", "rows": 16384, "sequences": 24, "uneven": True, "heads": 32, "kv_heads": 8,
         "width": 128, "frames": 4096, "layout": "packed", "ragged": True, "masked": False, "type": "bfloat16"},
        # one row through a layer's output projection: the weights' bytes
        {"name": "linear_row_one", "op": "linear", "rows": 1, "in": 5120, "out": 5120, "bias": True, "activation": "none",
         "residual": True, "eight": "none", "type": "bfloat16"},
        # the normed 8-bit rows of 64 streams into a feed-forward layer
        {"name": "linear_rows_e4m3", "op": "linear", "rows": 64, "in": 5120, "out": 10240, "bias": True,
         "activation": "silu", "residual": False, "eight": "e4m3", "type": "bfloat16"},
        # the stack's output rows of 32 windows to keys and values, 32 bits
        {"name": "linear_frames_fp32", "op": "linear", "rows": 18848, "in": 256, "out": 512, "bias": True,
         "activation": "leaky_relu", "residual": False, "eight": "none", "type": "float32"},
        # odd sizes: no two rows share an alignment
        {"name": "linear_odd_fp16", "op": "linear", "rows": 1111, "in": 777, "out": 999, "bias": True, "activation": "gelu",
         "residual": True, "eight": "none", "type": "float16"},
        # a prompt's rows through an output projection
        {"name": "linear_prompt", "op": "linear", "rows": 8192, "in": 5120, "out": 5120, "bias": True, "activation": "none",
         "residual": True, "eight": "none", "type": "bfloat16"},
        # the same from the norm's 8-bit rows
        {"name": "linear_prompt_e4m3", "op": "linear", "rows": 8192, "in": 5120, "out": 5120, "bias": True,
         "activation": "gelu", "residual": False, "eight": "e4m3", "type": "bfloat16"},
    ]


def _spread(rng, low, high):
    """A whole number of low..high, spread over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["cross_step", "cross", "cross", "linear", "linear", "linear"])
    case = {"op": op, "type": rng.choice(["float32", "bfloat16", "bfloat16", "float16"])}
    slow = 16 if case["type"] == "float32" else 1
    if op == "linear":
        case["eight"] = "none" if case["type"] == "float32" else rng.choice(["none", "none", "e4m3", "int8"])
        case["in"] = _spread(rng, 16, 8192)
        case["out"] = _spread(rng, 8, 8192)
        case["rows"] = min(_spread(rng, 1, 18848), max(1, int(MOST_PRODUCT / slow / (2 * case["in"] * case["out"]))))
        case["bias"] = rng.random() < 0.7
        case["activation"] = rng.choice(["none", "none", "relu", "leaky_relu", "gelu", "silu"])
        case["residual"] = rng.random() < 0.5
        return case
    case["kv_heads"] = rng.choice([1, 2, 4, 8, 16])
    case["heads"] = case["kv_heads"] * rng.choice([1, 1, 2, 4, 8 if case["kv_heads"] < 8 else 1])
    case["width"] = rng.choice([32, 64, 64, 80, 128, 128, 256])
    case["frames"] = _spread(rng, 1, 4096)
    case["layout"] = rng.choice(["padded", "packed"])
    case["ragged"] = rng.random() < 0.7
    case["masked"] = rng.random() < 0.3
    per_place = 2 * case["frames"] * case["kv_heads"] * case["width"]
    count = max(1, min(_spread(rng, 1, 256), int(MOST_MEMORY / per_place) - 2))
    if op == "cross_step":
        case["rows"] = count
        return case
    case["sequences"] = min(count, 32)
    most = int(MOST_ATTENTION / 2 / slow / (4 * case["frames"] * case["heads"] * case["width"]))
    case["rows"] = max(case["sequences"], min(_spread(rng, 1, 16384), most))
    case["uneven"] = rng.random() < 0.7
    return case


def _shares(total, count, uneven, seed):
    """Whole lengths that sum up to `total`: equal ones, or unequal ones with an empty one where there are three or more."""
    if not uneven or count == 1:
        return [total // count + (1 if i < total % count else 0) for i in range(count)]
    rng = random.Random(seed)
    cuts = sorted(rng.randint(0, total) for _ in range(count - (2 if count >= 3 else 1)))
    lengths = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    if count >= 3:
        lengths.insert(rng.randint(0, len(lengths)), 0)
    return lengths


def _lengths(case):
    """Rows of every sequence and frames of its memory: up to `frames`, unequal where ragged."""
    if case["op"] == "cross_step":
        rows = [1] * case["rows"]
    else:
        rows = _shares(case["rows"], case["sequences"], case["uneven"], 7 * case["rows"] + case["sequences"])
    most = case["frames"]
    rng = random.Random(case["rows"] + 1000003 * most)
    return rows, [rng.randint((most + 3) // 4, most) if case["ragged"] else most for _ in rows]


def work(case):
    size = 4 if case["type"] == "float32" else 2
    if case["op"] == "linear":
        m, k, n = case["rows"], case["in"], case["out"]
        part = 1 if case["eight"] != "none" else size
        moved = (m * k + n * k) * part + m * n * size * (2 if case["residual"] else 1) + n * size * case["bias"]
        return {"bytes": moved + (4 * (m + n) if part == 1 else 0), "flops": 2 * m * k * n}
    rows, frames = _lengths(case)
    inner, shared = case["heads"] * case["width"], case["kv_heads"] * case["width"]
    read = sum(f for r, f in zip(rows, frames) if r)
    return {"bytes": (2 * case["rows"] * inner + 2 * read * shared) * size + (read if case["masked"] else 0),
            "flops": 4 * inner * sum(r * f for r, f in zip(rows, frames))}


def prepare(case, seed):
    dtype = TYPES[case["type"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, kind=dtype):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(kind)

    def whole(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    s = dict(case)
    if case["op"] == "linear":
        m, k, n = case["rows"], case["in"], case["out"]
        s["x"], s["weight"] = normal(m, k), normal(n, k, scale=1 / math.sqrt(k))
        s["x_scales"] = s["weight_scales"] = None
        if case["eight"] != "none":  # a scale a row, as the norm gives its 8-bit rows
            code, top = EIGHT[case["eight"]]
            for name in ("x", "weight"):
                rows = s[name].float()
                scale = (rows.abs().amax(1) / top).clamp(min=1e-20)
                rows = (rows / scale[:, None]).clamp(-top, top)
                s[name] = rows.to(code) if case["eight"] == "e4m3" else torch.round(rows).to(code)
                s[name + "_scales"] = scale
        s["bias"] = normal(n) if case["bias"] else None
        s["residual"] = normal(m, n, scale=2.0) if case["residual"] else None
        return s
    rows, frames = _lengths(case)
    count, places = len(rows), len(rows) + 2
    # memories lie in a shuffled order, and some are read by no sequence
    order = torch.randperm(places, generator=g, device="cuda").tolist()
    held = [case["frames"]] * places
    for j in range(count):
        held[order[j]] = frames[j]
    size = [case["frames"]] * places if case["layout"] == "padded" else held
    starts = [0]
    for f in size:
        starts.append(starts[-1] + f)
    shared = case["kv_heads"] * case["width"]
    # keys and values lie side by side in one projection's rows
    s["kv"] = normal(starts[-1], 2 * shared)
    s["k"] = s["kv"][:, :shared].view(starts[-1], case["kv_heads"], case["width"])
    s["v"] = s["kv"][:, shared:].view(starts[-1], case["kv_heads"], case["width"])
    s["q"] = normal(sum(rows), case["heads"], case["width"], scale=2.0)
    s["slots"], s["memory_starts"] = whole(order[:count]), whole(starts)
    s["memory_lengths"] = whole(held) if case["layout"] == "padded" and case["ragged"] else None
    s["mask"] = torch.rand(starts[-1], generator=g, device="cuda") < 0.8 if case["masked"] else None
    bounds = [0]
    for r in rows:
        bounds.append(bounds[-1] + r)
    s["starts"] = whole(bounds) if case["op"] == "cross" else None
    s["most_rows"], s["most_frames"] = max(rows), max(frames)
    return s


# ---- the plain forms -------------------------------------------------------------------


def _plain_cross(s):
    """Runs of rows that never cross a sequence against their padded memories: a product, a softmax, a product."""
    q, dev = s["q"], s["q"].device
    rows, h, d = q.shape
    groups, per = s["kv_heads"], s["heads"] // s["kv_heads"]
    step = s["starts"] is None
    starts = torch.arange(rows + 1, device=dev) if step else s["starts"].long()
    count, size = starts.shape[0] - 1, min(RUN, s["most_rows"])
    # run i belongs to the sequence j with base[j] <= i < base[j + 1]; some runs are empty
    base = starts // size + (0 if step else torch.arange(count + 1, device=dev))
    i = torch.arange(rows // size + (0 if step else count), device=dev)
    sequence = torch.searchsorted(base[1:], i, right=True)
    token = (starts[sequence] + (i - base[sequence]) * size)[:, None] + torch.arange(size, device=dev)
    inside = token < starts[sequence + 1][:, None]
    token = torch.where(inside, token, 0)
    place = s["slots"].long()
    first, held = s["memory_starts"].long()[place], (s["memory_starts"][1:] - s["memory_starts"][:-1]).long()[place]
    if s["memory_lengths"] is not None:
        held = s["memory_lengths"].long()[place]
    at = torch.arange(s["most_frames"], device=dev)
    counts = at < held[:, None]
    frame = torch.where(counts, first[:, None] + at, 0)  # [sequences, frames]
    if s["mask"] is not None:
        counts = counts & s["mask"][frame]
    k = s["k"][frame].float().permute(0, 2, 3, 1)[sequence].contiguous()  # [runs, groups, d, frames]
    v = s["v"][frame].float().transpose(1, 2)[sequence].contiguous()  # [runs, groups, frames, d]
    qs = q[token].float().view(-1, size, groups, per, d).permute(0, 2, 3, 1, 4).reshape(-1, groups, per * size, d)
    score = torch.matmul(qs, k) * (1 / math.sqrt(d))
    keep = counts[sequence][:, None, None, :]
    score = torch.where(keep, score, float("-inf"))
    most = score.amax(3, keepdim=True)
    e = torch.exp(score - torch.where(most == float("-inf"), 0.0, most))
    total = e.sum(3, keepdim=True)
    y = torch.matmul(e, v) / torch.where(total > 0, total, 1.0)
    y = y.view(-1, groups, per, size, d).permute(0, 3, 1, 2, 4).reshape(-1, size, h, d)
    out = torch.empty(rows, h, d, device=dev)
    out[token[inside]] = y[inside]
    return {"y": out.to(q.dtype)}


def _activated(v, kind):
    if kind == "relu":
        return torch.clamp(v, min=0)
    if kind == "leaky_relu":
        return torch.where(v > 0, v, v * SLOPE)
    if kind == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if kind == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _plain_linear(s):
    v = torch.matmul(s["x"].float(), s["weight"].float().t())
    if s["x_scales"] is not None:
        v = v * s["x_scales"][:, None] * s["weight_scales"]
    if s["bias"] is not None:
        v = v + s["bias"].float()
    v = _activated(v, s["activation"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return {"y": v.to(TYPES[s["type"]])}


# ---- the package's entry points --------------------------------------------------------


def _own(s):
    import bidirectional_lstm_sequence_amd as bl

    if s["op"] == "linear":
        return {"y": bl.linear(s["x"], s["weight"], bias=s["bias"], residual=s["residual"], slope=SLOPE,
                               activation=None if s["activation"] == "none" else s["activation"],
                               x_scales=s["x_scales"], weight_scales=s["weight_scales"], out_type=TYPES[s["type"]])}
    if s["op"] == "cross_step":
        return {"y": bl.cross_attention_step(s["q"], s["k"], s["v"], s["memory_starts"], slots=s["slots"],
                                             memory_lengths=s["memory_lengths"], mask=s["mask"])}
    return {"y": bl.cross_attention(s["q"], s["k"], s["v"], s["starts"], s["memory_starts"], slots=s["slots"],
                                    memory_lengths=s["memory_lengths"], mask=s["mask"])}


def run(state):
    if own:
        return _own(state)
    return _plain_linear(state) if state["op"] == "linear" else _plain_cross(state)


# ---- 64 bits, from the definitions -----------------------------------------------------


def _exact_linear(s):
    x, w = s["x"].double(), s["weight"].double()
    if s["eight"] != "none":
        x, w = x * s["x_scales"].double()[:, None], w * s["weight_scales"].double()[:, None]
    v = torch.matmul(x, w.t().contiguous())
    if s["bias"] is not None:
        v += s["bias"].double()
    kind = s["activation"]
    if kind == "relu":
        v = torch.relu(v)
    elif kind == "leaky_relu":
        v = torch.nn.functional.leaky_relu(v, SLOPE)
    elif kind == "gelu":
        v = torch.nn.functional.gelu(v)
    elif kind == "silu":
        v = v * torch.sigmoid(v)
    return {"y": v if s["residual"] is None else v + s["residual"].double()}


def _exact_cross(s, case):
    """One sequence and one head of keys and values at a time."""
    rows, frames = _lengths(case)
    per, d = s["heads"] // s["kv_heads"], s["width"]
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for j, (r, f) in enumerate(zip(rows, frames)):
        first = int(s["memory_starts"][int(s["slots"][j])])
        chosen = slice(first, first + f) if s["mask"] is None else first + torch.nonzero(s["mask"][first: first + f])[:, 0]
        for g in range(s["kv_heads"] if r else 0):
            k, v = s["k"][chosen, g].double(), s["v"][chosen, g].double()
            if k.shape[0] == 0:
                continue
            q = s["q"][at: at + r, g * per: (g + 1) * per].double().reshape(r * per, d)
            weight = torch.softmax(torch.matmul(q, k.t().contiguous()) / math.sqrt(d), 1)
            y[at: at + r, g * per: (g + 1) * per] = torch.matmul(weight, v).view(r, per, d)
        at += r
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_linear(s) if case["op"] == "linear" else _exact_cross(s, case)
