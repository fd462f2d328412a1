"""Cases of the paged-cache operators that serve rotary, 4-bit and block-sparse attention, with their plain forms.

Five operators, each reached through the package's own entry points:

* ``rope``    keys and values appended to the paged cache with the position rotation applied on the way,
              the queries of the same tokens rotated by the same call (``pa_cache_append_rope``);
* ``append4`` the same rows appended to a cache held in 4 bits and read back as 16-bit rows
              (``pa_cache_append_q4``, ``pa_cache_read_q4``);
* ``decode4`` single-query attention over the 4-bit cache (``pa_decode_q4``);
* ``bounds``  the smallest and largest key of each frame, kept beside the cache (``pa_block_bounds``);
* ``sparse``  the frames that a score from those bounds selects for each query, and attention over
              them (``pa_select_blocks``, ``pa_decode_selected``).

A 4-bit row of D elements is D/2 bytes of codes (element 2i in the low half of byte i) and, for each
group of 32 elements, two fp16 numbers (step, offset): 5 bits an element.  A code n stands for the
fp16 number nearest to step * n + offset.
"""

import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
GROUP = 32
TOP = 65024.0  # 15 steps above the least value stay below what fp16 holds


# ---- cases ------------------------------------------------------------------------------------------


def listed():
    return [
        # a decode step of 64 sequences, 32 heads of 128: one new token each
        {"name": "rope step 64", "op": "rope", "seqs": 64, "count": 1, "hq": 32, "h": 32, "d": 128, "b": 16, "dtype": "f16",
         "rot": 128, "interleaved": False, "max_pos": 4096},
        # a chunked prefill batch: 16 chunks of 512 tokens, shared key heads
        {"name": "rope chunk 16x512", "op": "rope", "seqs": 16, "count": 512, "hq": 32, "h": 8, "d": 128, "b": 16, "dtype": "bf16",
         "rot": 128, "interleaved": False, "max_pos": 32768},
        # the decode step's append into the 4-bit cache
        {"name": "append4 step 64", "op": "append4", "seqs": 64, "count": 1, "hq": 32, "h": 32, "d": 128, "b": 16, "dtype": "f16",
         "rot": 128, "interleaved": False, "max_pos": 4096},
        # the chunked prefill batch's append into the 4-bit cache
        {"name": "append4 chunk 16x512", "op": "append4", "seqs": 16, "count": 512, "hq": 32, "h": 8, "d": 128, "b": 16,
         "dtype": "bf16", "rot": 128, "interleaved": False, "max_pos": 32768},
        # one user's chat: the latency of a short single sequence
        {"name": "decode4 1x1000", "op": "decode4", "seqs": 1, "lo": 1000, "hi": 1000, "hq": 32, "h": 8, "d": 128, "b": 16,
         "dtype": "bf16"},
        # the decode batch: 64 sequences of 512 to 2048 tokens
        {"name": "decode4 64x512-2048", "op": "decode4", "seqs": 64, "lo": 512, "hi": 2048, "hq": 32, "h": 32, "d": 128, "b": 16,
         "dtype": "f16"},
        # long contexts, few sequences: the context is split
        {"name": "decode4 4x16384", "op": "decode4", "seqs": 4, "lo": 16384, "hi": 16384, "hq": 32, "h": 32, "d": 128, "b": 16,
         "dtype": "bf16"},
        # the decode batch's step: the tail frame of each sequence
        {"name": "bounds step 64", "op": "bounds", "seqs": 64, "lo": 512, "hi": 2048, "count": 1, "h": 32, "d": 128, "b": 16,
         "dtype": "f16"},
        # after a prefill of 16 prompts: every frame
        {"name": "bounds prompt 16x4096", "op": "bounds", "seqs": 16, "lo": 4096, "hi": 4096, "count": 4096, "h": 8, "d": 128, "b": 32,
         "dtype": "bf16"},
        # one sequence of 8192 tokens, 512 of them attended
        {"name": "sparse 1x8192", "op": "sparse", "seqs": 1, "lo": 8192, "hi": 8192, "hq": 32, "h": 8, "d": 128, "b": 16,
         "dtype": "f16", "k": 32, "keep_first": 1, "keep_last": 2},
        # the long contexts, 1024 tokens of each attended by each head
        {"name": "sparse 4x16384", "op": "sparse", "seqs": 4, "lo": 16384, "hi": 16384, "hq": 32, "h": 32, "d": 128, "b": 16,
         "dtype": "bf16", "k": 64, "keep_first": 1, "keep_last": 2},
        # a ragged batch: short sequences beside very long ones, shared key heads
        {"name": "sparse 32x100-65536", "op": "sparse", "seqs": 32, "lo": 100, "hi": 65536, "hq": 32, "h": 8, "d": 128, "b": 32,
         "dtype": "f16", "k": 64, "keep_first": 1, "keep_last": 2},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "append4", "decode4", "decode4", "bounds", "sparse", "sparse"))
    d = rng.choice((64, 128, 128))
    h = rng.choice((1, 2, 4, 5, 8, 8, 16, 32))
    group = rng.choice([g for g in (1, 1, 2, 3, 4, 8, 16) if g * h <= 64])
    case = {"op": op, "h": h, "d": d, "b": rng.choice((8, 16, 16, 32, 64)), "dtype": rng.choice(("f16", "bf16"))}
    if op in ("rope", "append4"):
        seqs = _log(rng, 1, 200)
        case.update(seqs=seqs, count=_log(rng, 1, max(1, min(2048, 200000 // (seqs * h), 8192 // seqs))), hq=h * group,
                    rot=rng.choice((d, d, d // 2)), interleaved=rng.random() < 0.3, max_pos=32768)
    elif op == "bounds":
        seqs = _log(rng, 1, 200)
        hi = _log(rng, 2, max(2, min(30000, 500000 // (seqs * h))))
        case.update(seqs=seqs, lo=max(1, hi // rng.choice((1, 2, 10))), hi=hi, count=rng.choice((1, 1, 17, 30000)))
    else:
        seqs = _log(rng, 1, 100)
        hi = _log(rng, 2, max(2, min(65536, 2000000 // (seqs * h))))
        case.update(seqs=seqs, lo=max(1, hi // rng.choice((1, 2, 10, 100))), hi=hi, hq=h * group)
        if op == "sparse":
            blocks = -(-hi // case["b"])
            case.update(k=min(256, max(4, _log(rng, 1, 2 * blocks))), keep_first=rng.choice((0, 1, 1)), keep_last=rng.choice((1, 2)))
    return case


def _lens(case):
    """The lengths of a case's sequences: spread over [lo, hi], over their logarithm where that spans more than ten times."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    if n == 1:
        return [hi]
    at = [i / (n - 1) for i in range(n)]
    if hi > 10 * lo:
        lens = [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * x))) for x in at]
    else:
        lens = [int(round(lo + (hi - lo) * x)) for x in at]
    random.Random(n).shuffle(lens)
    return lens


def _first(case, length):
    """The first token that a bounds case's call has to look at: its last `count` tokens are new."""
    return max(0, length - case["count"])


def work(case):
    op, h, d, b = case["op"], case["h"], case["d"], case["b"]
    row4 = d // 2 + d // 8
    if op in ("rope", "append4"):
        t, hq = case["seqs"] * case["count"], case["hq"]
        rows = t * h * d * 2 * 2  # k and v, read
        q = t * hq * d * 2 * 2  # read and written
        table = min(t, case["max_pos"]) * case["rot"] * 4 + t * 8
        if op == "rope":
            return {"bytes": 2 * rows + q + table, "flops": 3 * t * (h + hq) * case["rot"]}
        return {"bytes": 2 * rows + 2 * 2 * t * h * row4 + q + table, "flops": 3 * t * (h + hq) * case["rot"] + 8 * t * h * d}
    lens = _lens(case)
    if op == "bounds":
        blocks = [-(-n // b) - _first(case, n) // b for n in lens]
        tokens = [n - _first(case, n) // b * b for n in lens]
        return {"bytes": sum(tokens) * h * d * 2 + sum(blocks) * (h * d * 4 + 4), "flops": 2 * sum(tokens) * h * d}
    hq = case["hq"]
    ends = len(lens) * hq * d * 4
    if op == "decode4":
        return {"bytes": sum(lens) * h * 2 * row4 + ends + sum(-(-n // b) for n in lens) * 4, "flops": 4 * sum(lens) * hq * d}
    blocks = [-(-n // b) for n in lens]
    tokens = [min(n, case["k"] * b) for n in lens]
    return {"bytes": sum(blocks) * (h * d * 4 + 4) + sum(tokens) * h * d * 4 + 2 * ends + len(lens) * h * case["k"] * 8,
            "flops": 2 * sum(blocks) * hq * d + 4 * sum(tokens) * hq * d}


# ---- inputs -----------------------------------------------------------------------------------------


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _keys(gen, shape, dtype):
    """Keys as a projection gives them: unit spread, with channels that sit away from zero."""
    d = shape[-1]
    centre = 2.0 * _randn(gen, shape[-2], d) * (torch.rand((shape[-2], d), generator=gen, device="cuda") < 0.1)
    return (_randn(gen, *shape) + centre).to(dtype)


def _tables(gen, lens, b):
    """Block tables over shuffled frames, and how many frames there are; entries behind a sequence's last are -1."""
    blocks = [-(-n // b) for n in lens]
    total = sum(blocks) + 7
    frames = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    width = max(blocks)
    at = torch.arange(width, device="cuda")
    count = torch.tensor(blocks, device="cuda")
    start = torch.cumsum(count, 0) - count
    index = (start[:, None] + at).clamp(max=total - 1)
    return torch.where(at < count[:, None], frames[index], torch.tensor(-1, dtype=torch.int32, device="cuda")).contiguous(), total


def _cos_sin(max_pos, rot):
    at = torch.arange(max_pos, device="cuda", dtype=torch.float64)
    rate = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = at[:, None] * rate
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()


def _prepare_append(case, gen):
    n, c, h, hq, d, b = (case[x] for x in ("seqs", "count", "h", "hq", "d", "b"))
    dtype = DTYPES[case["dtype"]]
    t = n * c
    per = -(-c // b) + 1  # frames of one sequence: it starts anywhere in its first one
    nb = n * per + 3
    frames = torch.randperm(nb, generator=gen, device="cuda")[: n * per].view(n, per)
    base = torch.randint(0, max(1, case["max_pos"] - c), (n, 1), generator=gen, device="cuda")
    pos = base + torch.arange(c, device="cuda")
    in_frames = base % b + torch.arange(c, device="cuda")
    slots = torch.gather(frames, 1, in_frames // b) * b + in_frames % b
    state = {
        "case": case, "k_new": _keys(gen, (t, h, d), dtype), "v_new": _randn(gen, t, h, d).to(dtype), "q": _randn(gen, t, hq, d).to(dtype),
        "slots": slots.reshape(-1).to(torch.int32), "positions": pos.reshape(-1).to(torch.int32),
        "cos_sin": _cos_sin(case["max_pos"], case["rot"]), "q_out": torch.empty((t, hq, d), dtype=dtype, device="cuda"),
    }
    if case["op"] == "rope":
        state["k_cache"], state["v_cache"] = (_randn(gen, nb, b, h, d).to(dtype) for _ in range(2))
    else:
        state["k_cache"], state["v_cache"] = (torch.zeros((nb, h, b, d // 2 + d // 8), dtype=torch.uint8, device="cuda") for _ in range(2))
        state["k_out"], state["v_out"] = (torch.empty((t, h, d), dtype=dtype, device="cuda") for _ in range(2))
    return state


def _pack(code, step, offset):
    """Rows of a 4-bit cache from codes [..., D] and fp16 numbers [..., D / 32]."""
    code = code.to(torch.uint8)
    params = torch.stack([step, offset], dim=-1).contiguous().view(torch.uint8).flatten(-2)
    return torch.cat([code[..., 0::2] | (code[..., 1::2] << 4), params], dim=-1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op in ("rope", "append4"):
        return _prepare_append(case, gen)
    h, d, b = case["h"], case["d"], case["b"]
    dtype = DTYPES[case["dtype"]]
    lens = _lens(case)
    tables, nb = _tables(gen, lens, b)
    state = {"case": case, "block_tables": tables, "context_lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
             "scale": d ** -0.5}
    if op == "decode4":
        for name in ("k_cache", "v_cache"):
            rows = _keys(gen, (nb, b, h, d), dtype) if name == "k_cache" else _randn(gen, nb, b, h, d).to(dtype)
            state[name] = _pack(*_quantise(rows.transpose(1, 2).float()))
    else:
        state["k_cache"] = _keys(gen, (nb, b, h, d), dtype)
        state["first"] = torch.tensor([_first(case, n) for n in lens] if op == "bounds" else [0] * len(lens), dtype=torch.int32, device="cuda")
        state["bounds"] = torch.zeros((nb, h, 2, d), dtype=dtype, device="cuda")
        if op == "sparse":
            state["v_cache"] = _randn(gen, nb, b, h, d).to(dtype)
            _bounds(state)  # a user's program keeps them beside the cache
            state["selected"] = torch.empty((len(lens), h, case["k"]), dtype=torch.int32, device="cuda")
    if op != "bounds":
        state["q"] = _randn(gen, len(lens), case["hq"], d).to(dtype)
        state["out"] = torch.empty_like(state["q"])
    return state


# ---- plain forms ------------------------------------------------------------------------------------


def _rotate(x, cos, sin, rot, interleaved):
    """x [T, H, D] in 32 bits with its first `rot` elements rotated, cos and sin [T, rot / 2]."""
    cos, sin, y = cos[:, None], sin[:, None], x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _rotated(state):
    case = state["case"]
    both = state["cos_sin"][state["positions"].long()]
    cos, sin = both[:, : case["rot"] // 2], both[:, case["rot"] // 2:]
    return [_rotate(state[x].float(), cos, sin, case["rot"], case["interleaved"]) for x in ("q", "k_new")]


def _quantise(x):
    """Codes [..., D], steps and offsets [..., D / 32] of rows x [..., D] in 32 bits."""
    x = x.clamp(-TOP, TOP).unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    offset = lo.half()
    step = ((hi - offset.float()) * (1.0 / 15.0)).half()
    code = torch.where(step > 0, ((x - offset.float()) / step.float()).round().clamp(0, 15), torch.zeros((), device=x.device))
    return code.flatten(-2), step[..., 0], offset[..., 0]


def _values(code, step, offset):
    """The numbers that codes [..., D] stand for, in 32 bits."""
    code = code.float().unflatten(-1, (-1, GROUP))
    return (code * step.float()[..., None] + offset.float()[..., None]).half().float().flatten(-2)


def _unpack(rows, d):
    code = torch.stack([rows[..., : d // 2] & 15, rows[..., : d // 2] >> 4], dim=-1).flatten(-2)
    params = rows[..., d // 2:].contiguous().view(torch.float16).unflatten(-1, (-1, 2))
    return code, params[..., 0], params[..., 1]


def _softmax_sum(scores, mask, v):
    """Weighted sums of v over the last axis of scores [..., N] where mask is true; zeros where it is nowhere."""
    scores = scores.masked_fill(~mask, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(scores - top)
    return (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _decode4(state):
    case = state["case"]
    s, h, d, b = case["seqs"], case["h"], case["d"], case["b"]
    frames = state["block_tables"].clamp(min=0).long()
    k, v = (_values(*_unpack(state[x][frames].transpose(1, 2).flatten(2, 3), d)) for x in ("k_cache", "v_cache"))  # [S, H, N, D]
    mask = torch.arange(k.shape[2], device="cuda") < state["context_lens"][:, None]
    q = state["q"].float().view(s, h, -1, d)
    out = _softmax_sum((q @ k.transpose(-1, -2)) * state["scale"], mask[:, None, None], v)
    return out.view(s, -1, d).to(state["q"].dtype)


def _bounds(state):
    """Bounds of the frames that hold each sequence's tokens from `first` on."""
    case, lens, first = state["case"], state["context_lens"].long(), state["first"].long()
    b, tables = case["b"], state["block_tables"].long()
    longest = max(-(-n // b) - (_first(case, n) // b if "count" in case else 0) for n in _lens(case))
    block = (first // b)[:, None] + torch.arange(longest, device="cuda")
    live = block * b < lens[:, None]
    frame = torch.gather(tables, 1, block.clamp(max=tables.shape[1] - 1))[live]
    inside = (block[..., None] * b + torch.arange(b, device="cuda") < lens[:, None, None])[live][..., None, None]
    k = state["k_cache"][frame]
    state["bounds"][frame, :, 0] = k.masked_fill(~inside, math.inf).amin(1)
    state["bounds"][frame, :, 1] = k.masked_fill(~inside, -math.inf).amax(1)
    return state["bounds"]


def _scores(state, bounds):
    """Scores [S, H, N] of each sequence's frames: for each query the largest product that a key within the bounds can give, the sum taken in
    32 bits over neighbours, then neighbours of those and so on; then the largest over the queries of a head."""
    case = state["case"]
    q = state["q"].float().view(case["seqs"], 1, case["h"], -1, case["d"])
    lo, hi = bounds[..., 0, :].float()[:, :, :, None], bounds[..., 1, :].float()[:, :, :, None]
    x = q * torch.where(q >= 0, hi, lo)
    while x.shape[-1] > 1:
        x = x[..., 0::2] + x[..., 1::2]
    return x[..., 0].amax(-1).transpose(1, 2)


def _sparse(state):
    case = state["case"]
    s, h, d, b, k = case["seqs"], case["h"], case["d"], case["b"], case["k"]
    lens, tables = state["context_lens"].long(), state["block_tables"].clamp(min=0).long()
    blocks = (lens + b - 1) // b
    at = torch.arange(tables.shape[1], device="cuda")
    keep = (at < case["keep_first"]) | (at >= (blocks - case["keep_last"])[:, None])
    score = _scores(state, state["bounds"][tables]).masked_fill(keep[:, None], math.inf)
    score = score.masked_fill((at >= blocks[:, None])[:, None], -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :k]
    none = torch.iinfo(torch.int32).max
    order = order.masked_fill(order >= blocks[:, None, None], none).sort(-1).values
    order = torch.nn.functional.pad(order, (0, k - order.shape[-1]), value=none)
    live = order < none
    token = order[..., None] * b + torch.arange(b, device="cuda")
    mask = (live[..., None] & (token < lens[:, None, None, None])).flatten(2)
    frame = torch.gather(tables[:, None].expand(s, h, -1), 2, order.clamp(max=tables.shape[1] - 1))
    heads = torch.arange(h, device="cuda")[None, :, None]
    kk, vv = (state[x][frame, :, heads].float().flatten(2, 3) for x in ("k_cache", "v_cache"))
    q = state["q"].float().view(s, h, -1, d)
    out = _softmax_sum((q @ kk.transpose(-1, -2)) * state["scale"], mask[:, :, None], vv)
    return {"out": out.view(s, -1, d).to(state["q"].dtype), "selected": order.masked_fill(~live, -1).to(torch.int32)}


def _plain(state):
    op = state["case"]["op"]
    if op in ("rope", "append4"):
        q, k = _rotated(state)
        dtype, slots = state["q"].dtype, state["slots"].long()
        if op == "rope":
            state["k_cache"].flatten(0, 1)[slots] = k.to(dtype)
            state["v_cache"].flatten(0, 1)[slots] = state["v_new"]
            return {"q": q.to(dtype), "k": state["k_cache"], "v": state["v_cache"]}
        return {"q": q.to(dtype), "k": _values(*_quantise(k)).to(dtype), "v": _values(*_quantise(state["v_new"].float())).to(dtype)}
    if op == "decode4":
        return {"out": _decode4(state)}
    if op == "bounds":
        return {"bounds": _bounds(state)}
    return _sparse(state)


# ---- the framework's calls --------------------------------------------------------------------------


def _own(s):
    import paged_kv_cache_126_gb300 as pa

    case = s["case"]
    op = case["op"]
    if op == "rope":
        pa.pa_cache_append_rope(s["k_new"], s["v_new"], s["slots"], s["k_cache"], s["v_cache"], s["positions"], s["cos_sin"],
                                q=s["q"], q_out=s["q_out"], interleaved=case["interleaved"])
        return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}
    if op == "append4":
        pa.pa_cache_append_q4(s["k_new"], s["v_new"], s["slots"], s["k_cache"], s["v_cache"], positions=s["positions"],
                              cos_sin=s["cos_sin"], q=s["q"], q_out=s["q_out"], interleaved=case["interleaved"])
        pa.pa_cache_read_q4(s["k_cache"], s["v_cache"], s["slots"], s["k_out"], s["v_out"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    if op == "decode4":
        pa.pa_decode_q4(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"], s["scale"], s["out"])
        return {"out": s["out"]}
    if op == "bounds":
        pa.pa_block_bounds(s["k_cache"], s["block_tables"], s["context_lens"], s["first"], s["bounds"])
        return {"bounds": s["bounds"]}
    pa.pa_select_blocks(s["q"], s["bounds"], s["block_tables"], s["context_lens"], case["b"], s["selected"],
                        keep_first=case["keep_first"], keep_last=case["keep_last"])
    pa.pa_decode_selected(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"], s["selected"], s["scale"], s["out"])
    return {"out": s["out"], "selected": s["selected"]}


def run(state):
    if own:
        return _own(state)
    else:
        return _plain(state)


# ---- the definitions in 64 bits -----------------------------------------------------------------------


def _turn64(x, angle_cos, angle_sin, rot, interleaved):
    """Rotation as a product of complex numbers."""
    x = x.double()
    z = x[..., :rot]
    z = torch.complex(z[..., 0::2], z[..., 1::2]) if interleaved else torch.complex(z[..., : rot // 2], z[..., rot // 2:])
    z = z * torch.complex(angle_cos.double(), angle_sin.double())[:, None]
    turned = torch.stack([z.real, z.imag], dim=-1).flatten(-2) if interleaved else torch.cat([z.real, z.imag], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _held64(x):
    """What rows x stand for once they are held in 4 bits."""
    parts = []
    for part in x.double().clamp(-TOP, TOP).split(GROUP, dim=-1):
        least = part.min(-1, keepdim=True).values.half().double()
        step = ((part.max(-1, keepdim=True).values - least) / 15).half().double()
        code = torch.zeros_like(part)
        code = torch.where(step == 0, code, torch.round((part - least) / torch.where(step == 0, torch.ones_like(step), step)).clip(0, 15))
        parts.append((least + code * step).half().double())
    return torch.cat(parts, dim=-1)


def _attend64(q, k, v, scale):
    """q [G, D] over k, v [N, D]."""
    return torch.softmax(scale * torch.einsum("gd,nd->gn", q, k), dim=-1) @ v if len(k) else torch.zeros_like(q)


def exact(case, seed):
    s = prepare(case, seed)
    op, h, d, b = case["op"], case["h"], case["d"], case["b"]
    if op == "bounds":
        got = s["bounds"].double()
        for i, n in enumerate(_lens(case)):
            for j in range(_first(case, n) // b, -(-n // b)) if case["seqs"] * n // b < 20000 else ():
                f = int(s["block_tables"][i, j])
                rows = s["k_cache"][f, : min(b, n - j * b)].double()
                got[f, :, 0], got[f, :, 1] = rows.min(0).values, rows.max(0).values
        return {"bounds": got} if case["seqs"] * case["hi"] // b < 20000 else None
    if op in ("rope", "append4"):
        table = s["cos_sin"].index_select(0, s["positions"])
        c, si = table.chunk(2, dim=1)
        q, k = (_turn64(s[x], c, si, case["rot"], case["interleaved"]) for x in ("q", "k_new"))
        if op == "append4":
            return {"q": q, "k": _held64(k), "v": _held64(s["v_new"])}
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        where = s["slots"].long()
        kc.view(-1, h, d).index_copy_(0, where, k)
        vc.view(-1, h, d).index_copy_(0, where, s["v_new"].double())
        return {"q": q, "k": kc, "v": vc}
    group = case["hq"] // h
    out = torch.zeros_like(s["q"], dtype=torch.float64)
    for i, n in enumerate(_lens(case)):
        count = -(-n // b)
        frames = s["block_tables"][i, :count].long()
        if op == "decode4":
            kv = []
            for x in ("k_cache", "v_cache"):
                rows = s[x][frames].permute(1, 0, 2, 3).reshape(h, count * b, -1)[:, :n]
                low, high = (rows[..., : d // 2] % 16).double(), (rows[..., : d // 2] // 16).double()
                fine = rows[..., d // 2:].contiguous().view(torch.half).double().repeat_interleave(GROUP, dim=-1).view(h, n, d // GROUP, 2, GROUP)
                code = torch.stack([low, high], -1).view(h, n, d // GROUP, GROUP)
                kv.append((fine[..., 0, :] * code + fine[..., 1, :]).half().double().view(h, n, d))
            for j in range(h):
                out[i, j * group:(j + 1) * group] = _attend64(s["q"][i, j * group:(j + 1) * group].double(), kv[0][j], kv[1][j], s["scale"])
            continue
        # the score's sum is one of 32 bits in a given order: the selection follows from that
        small, large = s["bounds"][frames, :, 0].float(), s["bounds"][frames, :, 1].float()  # [N, H, D]
        must = set(range(min(case["keep_first"], count))) | set(range(max(0, count - case["keep_last"]), count))
        for j in range(h):
            best = None
            for g in range(group):
                q = s["q"][i, j * group + g].float()
                part = torch.maximum(q * small[:, j], q * large[:, j])
                while part.shape[1] > 1:
                    part = part.view(count, -1, 2).sum(-1)
                best = part[:, 0] if best is None else torch.maximum(best, part[:, 0])
            rank = best.cpu().tolist()
            ranked = sorted(range(count), key=lambda x: (x not in must, 0.0 if x in must else -rank[x], x))
            take = torch.tensor(sorted(ranked[: case["k"]]), device="cuda")
            token = (take[:, None] * b + torch.arange(b, device="cuda")).flatten()
            token = token[token < n]
            kk, vv = (s[x][frames[token // b], token % b, j].double() for x in ("k_cache", "v_cache"))
            out[i, j * group:(j + 1) * group] = _attend64(s["q"][i, j * group:(j + 1) * group].double(), kk, vv, s["scale"])
    return {"out": out, "selected": None}
