"""Cases of the sequence operators: the short causal convolution, the selective state space scan,
the root-mean-square norm with an 8-bit output and the log probabilities of given tokens.

``run`` computes a case in plain torch operations (``own`` false) or through the package's entry
points (``own`` true); ``exact`` computes it in 64 bits, step by step from the definitions.
"""

import math

import torch

own = False

TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
CHUNK = 64  # steps of one chunk of the plain scan


def listed():
    return [
        # one new token of four streams through a layer's convolution: launch latency
        {"name": "conv_step_small", "op": "conv_step", "rows": 4, "channels": 4352, "taps": 4, "type": "bfloat16"},
        # 32 windows of 589 frames at the stack's output width plus two 64-wide projections
        {"name": "conv_frames_fp32", "op": "conv", "steps": 18848, "sequences": 32, "ragged": False, "carried": False,
         "channels": 384, "taps": 4, "type": "float32"},
        # a packed batch of prompts of unequal lengths, some continuing an earlier call
        {"name": "conv_prompts", "op": "conv", "steps": 16384, "sequences": 24, "ragged": True, "carried": True,
         "channels": 4352, "taps": 4, "type": "bfloat16"},
        # one new token of one stream
        {"name": "scan_step_one", "op": "scan_step", "rows": 1, "heads": 64, "width": 64, "groups": 1, "states": 128,
         "gated": True, "type": "bfloat16"},
        # one new token of 256 streams: the states' bytes
        {"name": "scan_step_many", "op": "scan_step", "rows": 256, "heads": 64, "width": 64, "groups": 1, "states": 128,
         "gated": True, "type": "bfloat16"},
        # 32 windows of 589 frames at the stack's output width, 32 bits
        {"name": "scan_frames_fp32", "op": "scan", "steps": 18848, "sequences": 32, "ragged": False, "carried": False,
         "heads": 4, "width": 64, "groups": 1, "states": 64, "gated": False, "type": "float32"},
        # one long prompt alone: few rows, the time axis has to be split
        {"name": "scan_one_prompt", "op": "scan", "steps": 4096, "sequences": 1, "ragged": False, "carried": False,
         "heads": 64, "width": 64, "groups": 1, "states": 128, "gated": True, "type": "bfloat16"},
        # a packed batch of prompts of unequal lengths, some continuing an earlier call
        {"name": "scan_prompts", "op": "scan", "steps": 16384, "sequences": 24, "ragged": True, "carried": True,
         "heads": 64, "width": 64, "groups": 1, "states": 128, "gated": True, "type": "bfloat16"},
        # the stack's output rows of 32 windows, added to a residual stream and normed in 32 bits
        {"name": "norm_frames_fp32", "op": "norm", "rows": 18848, "width": 256, "residual": True, "eight_bit": "none",
         "type": "float32"},
        # a prompt's rows on their way into an 8-bit projection
        {"name": "norm_wide_e4m3", "op": "norm", "rows": 8192, "width": 5120, "residual": True, "eight_bit": "e4m3",
         "type": "bfloat16"},
        # the heads' seven classes of 32 windows' frames: many tiny rows
        {"name": "logprobs_frames", "op": "logprobs", "rows": 18848, "tokens": 7, "given": 1, "top": 3, "type": "float32"},
        # a vocabulary of odd size, so that no two rows share an alignment
        {"name": "logprobs_vocabulary", "op": "logprobs", "rows": 512, "tokens": 100003, "given": 1, "top": 8,
         "type": "bfloat16"},
    ]


def _spread(rng, low, high):
    """A whole number of low..high, spread over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["conv_step", "conv", "scan_step", "scan", "scan", "norm", "logprobs"])
    case = {"op": op, "type": rng.choice(["float32", "bfloat16", "bfloat16", "float16"])}
    if op in ("conv", "conv_step"):
        case["channels"] = _spread(rng, 48, 4352)
        case["taps"] = rng.choice([2, 3, 4])
    if op in ("scan", "scan_step"):
        case["heads"] = _spread(rng, 1, 64)
        case["groups"] = rng.choice([g for g in (1, 2, 4, 8) if case["heads"] % g == 0])
        case["width"] = rng.choice([32, 64, 128])
        case["states"] = rng.choice([16, 32, 64, 128, 256])
        case["gated"] = rng.random() < 0.5
    if op in ("conv", "scan"):
        most = 16384
        if op == "conv" and case["type"] == "float32":
            most //= 2
        if op == "scan":
            most = min(most, 16384 * 64 * 64 * 128 // (case["heads"] * case["width"] * case["states"]))
            if case["type"] == "float32":
                most = max(1, most // 4)
        case["steps"] = _spread(rng, 1, most)
        case["sequences"] = _spread(rng, 1, min(32, case["steps"]))
        case["ragged"] = rng.random() < 0.7
        case["carried"] = rng.random() < 0.5
    if op == "conv_step":
        case["rows"] = _spread(rng, 1, 256)
    if op == "scan_step":
        case["rows"] = min(_spread(rng, 1, 256),
                           max(1, 256 * 64 * 64 * 128 // (case["heads"] * case["width"] * case["states"])))
    if op == "norm":
        case["width"] = _spread(rng, 32, 8192)
        case["rows"] = _spread(rng, 1, min(18848, 8192 * 5120 // (2 * case["width"])))
        case["residual"] = rng.random() < 0.7
        case["eight_bit"] = "none" if case["type"] == "float32" else rng.choice(["none", "e4m3", "int8"])
    if op == "logprobs":
        case["tokens"] = _spread(rng, 2, 131072)
        case["rows"] = _spread(rng, 1, min(18848, 512 * 100003 // (2 * case["tokens"])))
        case["given"] = rng.choice([1, 1, 2, 5])
        case["top"] = min(case["tokens"], rng.choice([0, 1, 3, 8, 20]))
    return case


def work(case):
    size = 4 if case["type"] == "float32" else 2
    op = case["op"]
    if op in ("conv", "conv_step"):
        rows = case["steps"] if op == "conv" else case["rows"]
        sequences = case["sequences"] if op == "conv" else case["rows"]
        kept = sequences * (case["taps"] - 1) * case["channels"]
        reads = kept if op == "conv_step" or case["carried"] else 0
        moved = 2 * rows * case["channels"] + kept + reads + case["channels"] * (case["taps"] + 1)
        return {"bytes": moved * size, "flops": rows * case["channels"] * (2 * case["taps"] + 4)}
    if op in ("scan", "scan_step"):
        rows = case["steps"] if op == "scan" else case["rows"]
        sequences = case["sequences"] if op == "scan" else case["rows"]
        inner = case["heads"] * case["width"]
        moved = rows * (inner * (3 if case["gated"] else 2) + case["heads"] + 2 * case["groups"] * case["states"]) * size
        state = sequences * inner * case["states"] * 4
        reads = op == "scan_step" or case["carried"]
        return {"bytes": moved + state * (2 if reads else 1) + case["heads"] * 12,
                "flops": rows * inner * case["states"] * 4}
    if op == "norm":
        n = case["rows"] * case["width"]
        out = {"none": size, "e4m3": 1, "int8": 1}[case["eight_bit"]]
        rest = case["rows"] * 4 if case["eight_bit"] != "none" else 0
        return {"bytes": n * (size * (3 if case["residual"] else 1) + out) + case["width"] * size + rest, "flops": 6 * n}
    n = case["rows"] * case["tokens"]
    return {"bytes": n * size + case["rows"] * (case["given"] * 12 + 4 + case["top"] * 12), "flops": 6 * n}


def _lengths(case, seed):
    """Lengths of the case's sequences: equal ones, or unequal ones with an empty one where there are three or more."""
    import random

    steps, count = case["steps"], case["sequences"]
    if not case["ragged"] or count == 1:
        return [steps // count + (1 if i < steps % count else 0) for i in range(count)]
    rng = random.Random(seed)
    cuts = sorted(rng.randint(0, steps) for _ in range(count - (2 if count >= 3 else 1)))
    lengths = [b - a for a, b in zip([0] + cuts, cuts + [steps])]
    if count >= 3:
        lengths.insert(rng.randint(0, len(lengths)), 0)
    return lengths


def prepare(case, seed):
    dtype = TYPES[case["type"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, kind=dtype):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(kind)

    def uniform(*shape, low=0.0, high=1.0):
        return torch.rand(*shape, generator=g, device="cuda") * (high - low) + low

    s = dict(case)
    op = case["op"]
    if op in ("conv", "scan"):
        lengths = _lengths(case, seed)
        starts = [0]
        for n in lengths:
            starts.append(starts[-1] + n)
        count = len(lengths)
        s["longest"] = max(lengths)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        # a cache with more places than sequences, taken in a shuffled order
        s["slots"] = torch.randperm(count + 3, generator=g, device="cuda")[:count].to(torch.int32)
        s["fresh"] = (uniform(count) < 0.5) if case["carried"] else torch.ones(count, dtype=torch.bool, device="cuda")
        rows = case["steps"]
    elif op in ("conv_step", "scan_step"):
        count = rows = case["rows"]
        s["slots"] = torch.randperm(count + 3, generator=g, device="cuda")[:count].to(torch.int32)
    if op in ("conv", "conv_step"):
        d, taps = case["channels"], case["taps"]
        s["x"] = normal(rows, d)
        s["weight"] = normal(d, taps, scale=1.0 / math.sqrt(taps))
        s["bias"] = normal(d, scale=0.1)
        s["state"] = normal(count + 3, taps - 1, d)
    if op in ("scan", "scan_step"):
        h, p, n, groups = case["heads"], case["width"], case["states"], case["groups"]
        # x, b and c lie side by side in the convolution's output rows
        s["xbc"] = normal(rows, h * p + 2 * groups * n, scale=0.7)
        s["x"] = s["xbc"][:, : h * p].view(rows, h, p)
        s["b"] = s["xbc"][:, h * p: h * p + groups * n].view(rows, groups, n)
        s["c"] = s["xbc"][:, h * p + groups * n:].view(rows, groups, n)
        s["dt"] = normal(rows, h, scale=0.5)
        step = torch.exp(uniform(h, low=math.log(1e-3), high=math.log(1e-1)))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus(dt_bias) = step
        s["a"] = -uniform(h, low=1.0, high=16.0)
        s["d"] = normal(h, scale=0.3, kind=torch.float32) + 1.0
        s["z"] = normal(rows, h, p) if case["gated"] else None
        s["state"] = normal(count + 3, h, p, n, scale=0.3, kind=torch.float32)
    if op == "norm":
        s["x"] = normal(case["rows"], case["width"])
        s["residual"] = normal(case["rows"], case["width"], scale=3.0) if case["residual"] else None
        s["weight"] = (uniform(case["width"], low=0.5, high=1.5)).to(dtype)
        s["eps"] = 1e-5
    if op == "logprobs":
        v = case["tokens"]
        s["logits"] = normal(case["rows"], v, scale=3.0)
        # a few tokens are masked away, never all of a row
        masked = torch.randint(0, v, (max(1, v // 50),), generator=g, device="cuda")
        if v > 8:
            s["logits"][:, masked] = float("-inf")
        s["ids"] = torch.randint(0, v, (case["rows"], case["given"]), generator=g, device="cuda")
    return s


# ---- the plain forms -------------------------------------------------------------------


def _plain_conv(s):
    x, taps, starts = s["x"], s["taps"], s["starts"].long()
    rows, dev = x.shape[0], x.device
    slots, w, d = s["slots"].long(), s["weight"].float(), s["channels"]
    sequence = torch.searchsorted(starts[1:], torch.arange(rows, device=dev), right=True)
    kept = s["state"][slots]
    kept = torch.where(s["fresh"][:, None, None], torch.zeros_like(kept), kept)
    # every sequence's W - 1 kept rows lie behind x's rows
    both = torch.cat([x, kept.reshape(-1, d)])

    def source(position, seq):  # rows of `both` at positions of sequences; negative ones are kept rows
        return torch.where(position >= 0, starts[seq] + position, rows + seq * (taps - 1) + taps - 1 + position)

    back = torch.arange(1 - taps, 1, device=dev)
    position = (torch.arange(rows, device=dev) - starts[sequence])[:, None] + back
    windows = both[source(position, sequence[:, None])].float()  # [rows, taps, channels]
    y = (windows * w.t()[None]).sum(1) + s["bias"].float()
    y = (y / (1 + torch.exp(-y))).to(x.dtype)
    lengths = starts[1:] - starts[:-1]
    each = torch.arange(lengths.shape[0], device=dev)
    last = both[source(lengths[:, None] + back[None, :-1], each[:, None])]
    # an empty sequence leaves its state as it was
    s["state"][slots] = torch.where((lengths > 0)[:, None, None], last, s["state"][slots])
    return {"y": y, "state": s["state"]}


def _plain_conv_step(s):
    x, slots = s["x"], s["slots"].long()
    window = torch.cat([s["state"][slots], x[:, None]], 1)
    y = (window.float() * s["weight"].float().t()[None]).sum(1) + s["bias"].float()
    s["state"][slots] = window[:, 1:]
    return {"y": (y / (1 + torch.exp(-y))).to(x.dtype), "state": s["state"]}


def _steps(dt, bias):
    v = dt.float() + bias
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _plain_scan(s):
    """Chunks of CHUNK steps, each within one sequence: products inside a chunk, and the chunks' states
    joined by a product with the decays between chunks. Logarithms of decays are summed in 64 bits."""
    x, starts, slots = s["x"], s["starts"].long(), s["slots"].long()
    rows, h, p = x.shape
    groups, n = s["groups"], s["states"]
    dev, count = x.device, starts.shape[0] - 1
    # chunk i belongs to the sequence j with base[j] <= i < base[j + 1]; some chunks are empty
    base = starts // CHUNK + torch.arange(count + 1, device=dev)
    chunks = rows // CHUNK + count
    i = torch.arange(chunks, device=dev)
    sequence = torch.searchsorted(base[1:], i, right=True)
    token = (starts[sequence] + (i - base[sequence]) * CHUNK)[:, None] + torch.arange(CHUNK, device=dev)
    inside = token < starts[sequence + 1][:, None]
    token = torch.where(inside, token, 0)
    step = torch.where(inside[:, :, None], _steps(s["dt"], s["dt_bias"])[token], 0.0)  # [chunks, L, h]
    decay = (step.double() * s["a"].double()).transpose(1, 2)  # [chunks, h, L]
    cum = torch.cumsum(decay, 2)
    xs = x[token].float().permute(0, 2, 1, 3).contiguous()  # [chunks, h, L, p]
    xdt = xs * step.transpose(1, 2)[..., None]
    b = s["b"][token].float().transpose(1, 2).contiguous()  # [chunks, groups, L, n]
    c = s["c"][token].float().transpose(1, 2).contiguous()
    per = h // groups
    # inside the chunk
    causal = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    between = torch.where(causal, cum[..., :, None] - cum[..., None, :], float("-inf")).float()
    cb = torch.matmul(c, b.transpose(2, 3).contiguous()).repeat_interleave(per, 1)
    y = torch.matmul(cb * torch.exp(between), xdt)
    # every chunk's own state, and what reaches its start from the chunks before it
    to_end = torch.exp((cum[..., -1:] - cum).float())
    weighted = (xdt * to_end[..., None]).transpose(2, 3).contiguous()  # [chunks, h, p, L]
    own_state = torch.matmul(weighted, b.repeat_interleave(per, 1)).reshape(chunks, h, p * n)
    total = cum[..., -1].t()  # [h, chunks]
    through = torch.cumsum(total, 1)
    earlier = (sequence[:, None] == sequence[None]) & (i[None] < i[:, None])
    reach = torch.exp(torch.where(earlier, (through - total)[:, :, None] - through[:, None, :], float("-inf")).float())
    arrived = torch.matmul(reach, own_state.transpose(0, 1).contiguous())  # [h, chunks, p * n]
    first = s["state"][slots]
    first = torch.where(s["fresh"][:, None, None, None], torch.zeros_like(first), first).reshape(count, h, p * n)
    before = through - total
    since = torch.exp((before - before[:, torch.clamp(base[sequence], max=chunks - 1)]).float())
    arrived = arrived + since[..., None] * first[sequence].transpose(0, 1)
    at = arrived.transpose(0, 1).reshape(chunks, h, p, n)
    carried = torch.matmul(c.repeat_interleave(per, 1), at.transpose(2, 3).contiguous())
    y = y + carried * torch.exp(cum.float())[..., None] + xs * s["d"][:, None, None]
    y = y.transpose(1, 2)  # [chunks, L, h, p]
    out = torch.empty(rows, h, p, device=dev)
    out[token[inside]] = y[inside]
    if s["z"] is not None:
        z = s["z"].float()
        out = out * (z / (1 + torch.exp(-z)))
    # the state behind each sequence's last chunk
    end = base[1:] - 1
    left = (at[end] * torch.exp(total[:, end].t().float())[..., None, None]
            + own_state.reshape(chunks, h, p, n)[end])
    empty = (starts[1:] == starts[:-1])[:, None, None, None]
    s["state"][slots] = torch.where(empty, s["state"][slots], left)
    return {"y": out.to(x.dtype), "state": s["state"]}


def _plain_scan_step(s):
    x, slots, per = s["x"].float(), s["slots"].long(), s["heads"] // s["groups"]
    step = _steps(s["dt"], s["dt_bias"])
    b = s["b"].float().repeat_interleave(per, 1)
    c = s["c"].float().repeat_interleave(per, 1)
    state = s["state"][slots] * torch.exp(step * s["a"])[..., None, None]
    state = state + (x * step[..., None])[..., None] * b[:, :, None, :]
    y = (state * c[:, :, None, :]).sum(3) + x * s["d"][:, None]
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z / (1 + torch.exp(-z)))
    s["state"][slots] = state
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


def _plain_norm(s):
    x = s["x"].float()
    total = x if s["residual"] is None else x + s["residual"].float()
    y = total * torch.rsqrt((total * total).mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
    got = {} if s["residual"] is None else {"residual": total.to(s["x"].dtype)}
    if s["eight_bit"] == "none":
        return {"y": y.to(s["x"].dtype), **got}
    most = y.abs().amax(1, keepdim=True)
    top = 448.0 if s["eight_bit"] == "e4m3" else 127.0
    scale = torch.where(most > 0, most / top, 1.0)
    if s["eight_bit"] == "e4m3":
        q = (y / scale).clamp(-top, top).to(torch.float8_e4m3fn)
    else:
        q = torch.round(y / scale).clamp(-top, top).to(torch.int8)
    return {**_eight(s, q), "scales": scale[:, 0], **({"values": _values(s, q, scale)} if s["eight_bit"] == "int8" else {}), **got}


def _eight(s, q):
    return {"q": q} if s["eight_bit"] == "e4m3" else {}


def _values(s, q, scale):
    """What int8 codes stand for, in the input's type."""
    return (q.float() * scale).to(s["x"].dtype)


def _order(z):
    """Whole numbers that order 32-bit floats, larger ones first, and of equal ones the lowest place first."""
    bits = (z + 0.0).view(torch.int32).long()
    bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    return bits * (1 << 20) - torch.arange(z.shape[1], device=z.device)


def _plain_logprobs(s):
    z = s["logits"].float()
    most = z.amax(1, keepdim=True)
    off = z - most
    e = torch.exp(off)
    total = e.sum(1, keepdim=True)
    rest = torch.log(total)
    entropy = rest[:, 0] - torch.where(e > 0, e * off, 0.0).sum(1) / total[:, 0]
    given = torch.gather(off, 1, s["ids"]) - rest
    got = {"logprobs": given, "entropy": entropy}
    if s["top"]:
        place = torch.topk(_order(z), s["top"], dim=1).indices
        got["top_tokens"] = place
        got["top_logprobs"] = torch.gather(off, 1, place) - rest
    return got


PLAIN = {"conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan, "scan_step": _plain_scan_step,
         "norm": _plain_norm, "logprobs": _plain_logprobs}


# ---- the package's entry points --------------------------------------------------------


def _own(s):
    import bidirectional_lstm_sequence_amd as bl

    op = s["op"]
    if op == "conv":
        y = bl.causal_conv(s["x"], s["weight"], s["starts"], bias=s["bias"], state=s["state"], slots=s["slots"],
                           fresh=s["fresh"])
        return {"y": y, "state": s["state"]}
    if op == "conv_step":
        y = bl.causal_conv_step(s["x"], s["weight"], s["state"], bias=s["bias"], slots=s["slots"])
        return {"y": y, "state": s["state"]}
    if op == "scan":
        y = bl.selective_scan(s["x"], s["dt"], s["a"], s["b"], s["c"], s["starts"], d=s["d"], z=s["z"],
                              dt_bias=s["dt_bias"], softplus=True, state=s["state"], slots=s["slots"], fresh=s["fresh"])
        return {"y": y, "state": s["state"]}
    if op == "scan_step":
        y = bl.selective_scan_step(s["x"], s["dt"], s["a"], s["b"], s["c"], s["state"], d=s["d"], z=s["z"],
                                   dt_bias=s["dt_bias"], softplus=True, slots=s["slots"])
        return {"y": y, "state": s["state"]}
    if op == "norm":
        r = bl.add_rms_norm(s["x"], s["weight"], s["eps"], residual=s["residual"],
                            eight_bit=None if s["eight_bit"] == "none" else s["eight_bit"])
        got = {} if s["residual"] is None else {"residual": r.residual}
        if s["eight_bit"] == "none":
            return {"y": r.y, **got}
        more = {"values": _values(s, r.q, r.scales[:, None])} if s["eight_bit"] == "int8" else {}
        return {**_eight(s, r.q), "scales": r.scales, **more, **got}
    r = bl.token_logprobs(s["logits"], s["ids"], top=s["top"])
    got = {"logprobs": r.logprobs, "entropy": r.entropy}
    if s["top"]:
        got.update(top_tokens=r.top_tokens, top_logprobs=r.top_logprobs)
    return got


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---- 64 bits, from the definitions -----------------------------------------------------


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _exact_conv(s, rows, lengths):
    """Each sequence as its kept rows followed by its own, tap by tap."""
    taps, w = s["taps"], s["weight"].double()
    y = torch.zeros(rows, s["channels"], dtype=torch.float64, device="cuda")
    state = s["state"].double()
    at = 0
    for j, length in enumerate(lengths):
        if length == 0:
            continue
        slot = int(s["slots"][j])
        head = torch.zeros_like(state[slot]) if "fresh" in s and bool(s["fresh"][j]) else state[slot]
        line = torch.cat([head, s["x"][at: at + length].double()])
        v = s["bias"].double().expand(length, -1)
        for k in range(taps):
            v = v + w[:, k] * line[k: k + length]
        y[at: at + length] = v * _sigmoid(v)
        state[slot] = line[length:]
        at += length
    return {"y": y, "state": state}


def _exact_scan(s, rows, lengths):
    """The recurrence, one step of all sequences at a time."""
    h, p, n, per = s["heads"], s["width"], s["states"], s["heads"] // s["groups"]
    dev = "cuda"
    count = len(lengths)
    length = torch.tensor(lengths, device=dev)
    starts = torch.cumsum(length, 0) - length
    slots = s["slots"].long()
    state = s["state"][slots].double()
    if "fresh" in s:
        state[s["fresh"] & (length > 0)] = 0
    y = torch.zeros(rows, h, p, dtype=torch.float64, device=dev)
    step = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=200)
    a = s["a"].double()
    order = torch.argsort(length, descending=True, stable=True)
    sizes = length[order].tolist()
    live = count
    for t in range(max(lengths)):
        while live and sizes[live - 1] <= t:
            live -= 1
        j = order[:live]
        token = starts[j] + t
        dt = step[token]
        b = s["b"][token].double().repeat_interleave(per, 1)
        c = s["c"][token].double().repeat_interleave(per, 1)
        x = s["x"][token].double()
        here = state[j] if live < count or count > 1 else state
        here = here * torch.exp(dt * a)[..., None, None] + (dt[..., None] * x)[..., None] * b[:, :, None, :]
        y[token] = torch.matmul(here, c[..., None])[..., 0] + s["d"].double()[:, None] * x
        if live < count or count > 1:
            state[j] = here
        else:
            state = here
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z * _sigmoid(z)
    kept = s["state"].double()
    kept[slots] = state
    return {"y": y, "state": kept}


def _exact_e4m3(v):
    """The nearest e4m3 value, ties to even: steps of 2^(e - 3), e the exponent, from 2^-9 on."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -60)))
    unit = torch.exp2(torch.clamp(e, min=-6) - 3)
    return (torch.round(v / unit) * unit).clamp(-448, 448)


def _exact_norm(s):
    total = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
    y = s["weight"].double() * total / torch.sqrt(total.pow(2).sum(1, keepdim=True) / s["width"] + s["eps"])
    got = {} if s["residual"] is None else {"residual": total}
    if s["eight_bit"] == "none":
        return {"y": y, **got}
    scale = y.abs().max(1, keepdim=True).values / (448.0 if s["eight_bit"] == "e4m3" else 127.0)
    if s["eight_bit"] == "e4m3":
        return {"q": _exact_e4m3(y / scale), "scales": scale[:, 0], **got}
    return {"scales": scale[:, 0], "values": torch.round(y / scale) * scale, **got}


def _exact_logprobs(s):
    logp = torch.log_softmax(s["logits"].double(), 1)
    got = {"logprobs": torch.gather(logp, 1, s["ids"]),
           "entropy": -torch.where(torch.isinf(logp), 0.0, torch.exp(logp) * logp).sum(1)}
    if s["top"]:
        got["top_tokens"] = None
        got["top_logprobs"] = torch.sort(logp, 1, descending=True).values[:, : s["top"]]
    return got


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(s)
    if op == "logprobs":
        return _exact_logprobs(s)
    if op in ("conv_step", "scan_step"):
        rows, lengths = case["rows"], [1] * case["rows"]
    else:
        rows, lengths = case["steps"], _lengths(case, seed)
    return (_exact_conv if op.startswith("conv") else _exact_scan)(s, rows, lengths)
