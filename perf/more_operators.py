"""Cases of the paged-cache operators that bound what a long context costs, with their plain forms.

Four operators, each reached through the package's own entry points:

* ``window``  single-query attention over a sequence's last tokens and its first few (``pa_decode_window``);
* ``chunk``   the same for chunks of queries, each of which sees its own last tokens (``pa_prefill_window``);
* ``append8`` keys and values appended to a cache held in 8 bits, one step per frame and head, and the frames that
              the call wrote to read back as 16-bit rows (``pa_cache_append_q8``, ``pa_cache_read_q8``);
* ``decode8`` single-query attention over the 8-bit cache, every token of it or a window (``pa_decode_q8``).

A query at position p sees the keys at j <= p with j > p - window or j < sinks; a window of 0 is every key (``decode8``).

A byte b of the 8-bit cache stands for (b - 128) * step, b >= 1, the step being that of its frame and head.  A frame that
begins with a call's tokens takes r = 127 / max |x| with all but its 8 leading bits cleared, and step = 1 / r; one that holds earlier
tokens keeps its step, or doubles it (and halves the earlier codes, ties to even) until the new tokens fit.
"""

import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
LEAST, MOST = 2.0 ** -60, 2.0 ** 60  # what a frame's largest element counts as, at least and at most


# ---- cases ------------------------------------------------------------------------------------------


def listed():
    return [
        # one user's long chat: the latency of a single sequence, 1024 tokens of it in sight
        {"name": "window 1x20000", "op": "window", "seqs": 1, "lo": 20000, "hi": 20000, "hq": 32, "h": 8, "d": 128, "b": 16,
         "dtype": "bf16", "window": 1024, "sinks": 4},
        # a decode batch of 64 sequences, some of them shorter than the window
        {"name": "window 64x512-16384", "op": "window", "seqs": 64, "lo": 512, "hi": 16384, "hq": 32, "h": 32, "d": 128, "b": 16,
         "dtype": "f16", "window": 1024, "sinks": 4},
        # a ragged batch, shared key heads, a wide window that begins inside a frame
        {"name": "window 32x100-65536", "op": "window", "seqs": 32, "lo": 100, "hi": 65536, "hq": 32, "h": 8, "d": 128, "b": 32,
         "dtype": "bf16", "window": 4000, "sinks": 4},
        # a chunk of one long prompt between decode steps
        {"name": "chunk 1x512", "op": "chunk", "seqs": 1, "count": 512, "lo": 8192, "hi": 8192, "hq": 32, "h": 8, "d": 128, "b": 16,
         "dtype": "bf16", "window": 1024, "sinks": 4},
        # the chunked prefill batch: 16 ragged chunks over prefixes of different lengths
        {"name": "chunk 16x512", "op": "chunk", "seqs": 16, "count": 512, "lo": 1, "hi": 8000, "hq": 32, "h": 32, "d": 128, "b": 16,
         "dtype": "f16", "window": 2048, "sinks": 4},
        # a whole prompt at once, shared key heads
        {"name": "chunk 1x16384", "op": "chunk", "seqs": 1, "count": 16384, "lo": 0, "hi": 0, "hq": 32, "h": 8, "d": 128, "b": 32,
         "dtype": "bf16", "window": 4096, "sinks": 0},
        # the decode step's append: one token each, most of them into frames that hold earlier ones
        {"name": "append8 step 64", "op": "append8", "seqs": 64, "count": 1, "lo": 512, "hi": 2048, "h": 32, "d": 128, "b": 16,
         "dtype": "f16"},
        # the chunked prefill batch's append
        {"name": "append8 chunk 16x512", "op": "append8", "seqs": 16, "count": 512, "lo": 1, "hi": 8000, "h": 8, "d": 128, "b": 16,
         "dtype": "bf16"},
        # one user's chat: the latency of a short single sequence
        {"name": "decode8 1x1000", "op": "decode8", "seqs": 1, "lo": 1000, "hi": 1000, "hq": 32, "h": 8, "d": 128, "b": 16,
         "dtype": "bf16", "window": 0, "sinks": 0},
        # the decode batch: 64 sequences of 512 to 2048 tokens
        {"name": "decode8 64x512-2048", "op": "decode8", "seqs": 64, "lo": 512, "hi": 2048, "hq": 32, "h": 32, "d": 128, "b": 16,
         "dtype": "f16", "window": 0, "sinks": 0},
        # long contexts, few sequences: the context is split
        {"name": "decode8 4x16384", "op": "decode8", "seqs": 4, "lo": 16384, "hi": 16384, "hq": 32, "h": 32, "d": 128, "b": 16,
         "dtype": "bf16", "window": 0, "sinks": 0},
        # both bounds together: a ragged batch's windows over the 8-bit cache
        {"name": "decode8 32x100-65536", "op": "decode8", "seqs": 32, "lo": 100, "hi": 65536, "hq": 32, "h": 8, "d": 128, "b": 32,
         "dtype": "f16", "window": 4000, "sinks": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("window", "window", "chunk", "chunk", "append8", "decode8", "decode8"))
    h = rng.choice((1, 2, 4, 5, 8, 8, 16, 32))
    group = rng.choice([g for g in (1, 1, 2, 3, 4, 8, 16) if g * h <= 64])
    case = {"op": op, "h": h, "d": rng.choice((64, 128, 128)), "b": rng.choice((8, 16, 16, 32, 64, 128)),
            "dtype": rng.choice(("f16", "bf16"))}
    spread = rng.choice((1, 2, 10, 100))
    if op == "append8":
        seqs = _log(rng, 1, 200)
        hi = _log(rng, 2, 20000)
        case.update(seqs=seqs, count=_log(rng, 1, max(1, min(2048, 65536 // (seqs * h), 8192 // seqs))), lo=hi // spread, hi=hi)
        return case
    case.update(hq=h * group, window=_log(rng, 1, 8192), sinks=rng.choice((0, 1, 4, 4, 16, 100)))
    if op == "chunk":
        seqs = _log(rng, 1, 40)
        count = _log(rng, 1, max(1, min(8192, 16384 // seqs)))
        hi = _log(rng, 1, 20000)
        case.update(d=128, seqs=seqs, count=count, lo=hi // spread, hi=hi)
        # no more pairs of query and key than the whole prompt of 16384 has
        case["window"] = max(1, min(case["window"], 2000000000 // (seqs * count * case["hq"])))
        return case
    if op == "decode8" and rng.random() < 0.5:
        case.update(window=0, sinks=0)
    seqs = _log(rng, 1, 100)
    hi = _log(rng, 2, 65536)
    if case["window"]:
        case["window"] = min(case["window"], max(1, 1500000 // (seqs * h)))
    else:
        hi = min(hi, max(2, 2000000 // (seqs * h)))
    case.update(seqs=seqs, lo=max(1, hi // spread), hi=hi)
    return case


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], over their logarithm where that spans more than ten times, in a fixed shuffled order."""
    if n == 1:
        return [hi]
    at = [i / (n - 1) for i in range(n)]
    if lo > 0 and hi > 10 * lo:
        out = [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * x))) for x in at]
    else:
        out = [int(round(lo + (hi - lo) * x)) for x in at]
    random.Random(n).shuffle(out)
    return out


def _lens(case):
    """(tokens, new ones among them) of each sequence of a case."""
    before = _spread(case["seqs"], case["lo"], case["hi"])
    if case["op"] not in ("chunk", "append8"):
        return [(n, 1) for n in before]
    fresh = _spread(case["seqs"], (case["count"] + 1) // 2, case["count"])[::-1]
    return [(n + c, c) for n, c in zip(before, fresh)]


def _start(case, p):
    """First token of the window of a query at position p."""
    return max(0, p + 1 - case["window"]) if case.get("window") else 0


def _seen(case, p):
    """Keys that a query at position p sees."""
    start = _start(case, p)
    return p + 1 - start + min(case.get("sinks", 0), start)


def _frames(case, length, fresh):
    """Positions in its table of the frames that a sequence's call reads or writes."""
    b, first = case["b"], length - fresh
    start = first if case["op"] == "append8" else _start(case, first)
    sinks = 0 if case["op"] == "append8" else min(case["sinks"], start)
    return sorted(set(range(-(-sinks // b))) | set(range(start // b, -(-length // b))))


def work(case):
    op, h, d = case["op"], case["h"], case["d"]
    lens = _lens(case)
    frames = sum(len(_frames(case, n, c)) for n, c in lens)
    if op == "append8":
        rows = sum(c for _, c in lens)
        held = sum(n - (n - c) // case["b"] * case["b"] for n, c in lens)  # tokens of the frames written to, read back
        return {"bytes": rows * h * d * 2 * (2 + 1) + held * h * d * 2 * (1 + 2) + frames * (h * 8 * 2 + 4),
                "flops": rows * h * d * 2 * 2 + held * h * d * 2}
    hq = case["hq"]
    rows = sum(c for _, c in lens)
    pairs, keys = 0, 0
    for n, c in lens:
        keys += n - _start(case, n - c) + min(case["sinks"], _start(case, n - c))
        pairs += sum(_seen(case, p) for p in range(n - c, n))
    size = 2 * h * d * (1 if op == "decode8" else 2)
    return {"bytes": keys * size + rows * hq * d * 4 + frames * 4 + (frames * h * 8 if op == "decode8" else 0), "flops": 4 * pairs * hq * d}


# ---- inputs -----------------------------------------------------------------------------------------


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _keys(gen, shape, dtype):
    """Keys as a projection gives them: unit spread, with channels that sit away from zero."""
    d = shape[-1]
    centre = 2.0 * _randn(gen, shape[-2], d) * (torch.rand((shape[-2], d), generator=gen, device="cuda") < 0.1)
    return (_randn(gen, *shape) + centre).to(dtype)


def _tables(gen, case, lens):
    """Block tables over shuffled frames, and how many frames there are: those that no query sees are given up (-1), as are the
    entries behind a sequence's last."""
    held = [_frames(case, n, c) for n, c in lens]
    total = sum(len(x) for x in held) + 7
    frames = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    at = torch.tensor([j for x in held for j in x], device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor([len(x) for x in held], device="cuda"))
    tables = torch.full((len(lens), max(-(-n // case["b"]) for n, _ in lens)), -1, dtype=torch.int32, device="cuda")
    tables[seq, at] = frames[: len(at)]
    return tables, total


def _frames8(gen, case, nb, keys):
    """An 8-bit cache whose frames were each filled by one append, and its steps."""
    h, d, b, dtype = case["h"], case["d"], case["b"], DTYPES[case["dtype"]]
    cache = torch.empty((nb, h, b, d), dtype=torch.uint8, device="cuda")
    step = torch.empty((nb, h), dtype=torch.float32, device="cuda")
    for i in range(0, nb, 2048):
        n = min(2048, nb - i)
        x = (_keys(gen, (n, b, h, d), dtype) if keys else _randn(gen, n, b, h, d).to(dtype)).float().transpose(1, 2)
        r = _rate(x.abs().amax((-1, -2)))
        cache[i:i + n] = _codes(x, r[..., None, None])
        step[i:i + n] = torch.ones_like(r) / r
    return cache, step


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, h, d, b = case["op"], case["h"], case["d"], case["b"]
    dtype = DTYPES[case["dtype"]]
    lens = _lens(case)
    tables, nb = _tables(gen, case, lens)
    start = [0]
    for _, c in lens:
        start.append(start[-1] + c)
    whole = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    state = {"case": case, "block_tables": tables, "context_lens": whole([n for n, _ in lens]), "query_start": whole(start),
             "scale": d ** -0.5}
    if op in ("window", "chunk"):
        state["k_cache"], state["v_cache"] = _keys(gen, (nb, b, h, d), dtype), _randn(gen, nb, b, h, d).to(dtype)
    else:
        state["k_cache"], state["k_scale"] = _frames8(gen, case, nb, True)
        state["v_cache"], state["v_scale"] = _frames8(gen, case, nb, False)
    if op == "append8":
        state["k_new"], state["v_new"] = _keys(gen, (start[-1], h, d), dtype), _randn(gen, start[-1], h, d).to(dtype)
        state["slots"] = torch.cat([(tables[i, (n - c) // b: -(-n // b), None].long() * b + torch.arange(b, device="cuda")).flatten()
                                    [: n - (n - c) // b * b] for i, (n, c) in enumerate(lens)]).to(torch.int32)
        state["k_out"], state["v_out"] = (torch.empty((len(state["slots"]), h, d), dtype=dtype, device="cuda") for _ in range(2))
    else:
        state["q"] = _randn(gen, start[-1], case["hq"], d).to(dtype)
        state["out"] = torch.empty_like(state["q"])
    return state


# ---- plain forms ------------------------------------------------------------------------------------


def _rate(largest):
    """Codes per unit of a frame whose largest element is `largest`: 127 / largest, all but its 8 leading bits cleared."""
    r = torch.full_like(largest, 127.0) / largest.clamp(LEAST, MOST)
    return (r.view(torch.int32) & -65536).view(torch.float32)


def _codes(x, r):
    """Bytes of x: products of at most 19 bits, so that the rounding to whole numbers is the only one."""
    return ((x * r).round().clamp(-127, 127) + 128).to(torch.uint8)


def _fill(state, name, frame, row, fresh, old):
    """Rows `row` [F, B] of the new tokens, where `fresh` [F, B], into frames [F] of one cache; `old` [F, B]: earlier tokens."""
    cache, step = state[name + "_cache"], state[name + "_scale"]
    x = state[name + "_new"][row].float().transpose(1, 2)  # [F, H, B, D]
    fresh, old = fresh[:, None, :, None], old[:, None, :, None]
    largest = x.abs().masked_fill(~fresh, 0.0).amax((-1, -2)).clamp(LEAST, MOST)
    begun = old.any(2)[..., 0]  # [F, 1]
    was = step[frame]
    kept = (torch.ones_like(was) / was).to(torch.bfloat16).float()  # the rate that the step is one over
    over = largest * kept
    more = (torch.frexp(over).exponent - 7).clamp(min=0)
    more = torch.where(torch.ldexp(over, -more) > 127, more + 1, more)
    r = torch.where(begun, torch.ldexp(kept, -more), _rate(largest))
    codes = cache[frame]
    halved = (torch.ldexp(codes.float() - 128, -more[..., None, None]).round() + 128).to(torch.uint8)
    cache[frame] = torch.where(fresh, _codes(x, r[..., None, None]), torch.where(old, halved, codes))
    step[frame] = torch.where(begun, torch.ldexp(was, more), torch.ones_like(r) / r)


def _append8(state):
    case, lens = state["case"], state["context_lens"].long()
    b, start = case["b"], state["query_start"].long()
    first = lens - (start[1:] - start[:-1])
    longest = max(-(-n // b) - (n - c) // b for n, c in _lens(case))
    block = (first // b)[:, None] + torch.arange(longest, device="cuda")
    seq, at = torch.nonzero(block * b < lens[:, None], as_tuple=True)
    block = block[seq, at]
    frame = state["block_tables"][seq, block].long()
    token = block[:, None] * b + torch.arange(b, device="cuda")
    old = token < first[seq, None]
    fresh = ~old & (token < lens[seq, None])
    row = torch.where(fresh, token - first[seq, None] + start[seq, None], torch.zeros_like(token))
    out = {}
    for name in ("k", "v"):
        _fill(state, name, frame, row, fresh, old)
        held = state["slots"].long()
        codes = state[name + "_cache"][held // b, :, held % b].float() - 128
        out[name] = (codes * state[name + "_scale"][held // b][..., None]).to(state["k_new"].dtype)
        out[name + "_scale"] = state[name + "_scale"]
    return out


def _softmax_sum(scores, mask, v):
    """Weighted sums of v over the last axis of scores [..., N] where mask is true; zeros where it is nowhere."""
    scores = scores.masked_fill(~mask, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(scores - top)
    return (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _decode(state):
    case, lens = state["case"], state["context_lens"].long()[:, None]
    s, h, d, b = case["seqs"], case["h"], case["d"], case["b"]
    most = max(_seen(case, n - 1) for n, _ in _lens(case))
    begin = (lens - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(lens)
    sinks = begin.clamp(max=case["sinks"])
    at = torch.arange(most, device="cuda")
    token = torch.where(at < sinks, at, at - sinks + begin)  # [S, N]
    mask = token < lens
    token = torch.minimum(token, lens - 1)
    frame = torch.gather(state["block_tables"], 1, token // b).long()
    rows = []
    for x in ("k", "v"):
        if case["op"] == "window":
            rows.append(state[x + "_cache"][frame, token % b].float().transpose(1, 2))  # [S, H, N, D]
        else:
            step = state[x + "_scale"][frame].transpose(1, 2)[..., None]
            rows.append((state[x + "_cache"][frame, :, token % b].float() - 128).transpose(1, 2) * step)
    q = state["q"].float().view(s, h, -1, d)
    out = _softmax_sum((q @ rows[0].transpose(-1, -2)) * state["scale"], mask[:, None, None], rows[1])
    return out.view(s, -1, d).to(state["q"].dtype)


def _chunk(state, block=512):
    """A block of queries at a time, against the keys that any of them sees."""
    case, row = state["case"], 0
    h, d, b = case["h"], case["d"], case["b"]
    out = torch.empty_like(state["q"])
    for i, (n, c) in enumerate(_lens(case)):
        for p0 in range(n - c, n, block):
            p1 = min(n, p0 + block)
            begin = _start(case, p0)
            token = torch.cat([torch.arange(min(case["sinks"], begin), device="cuda"), torch.arange(begin, p1, device="cuda")])
            frame = state["block_tables"][i, token // b].long()
            k, v = (state[x][frame, token % b].float().transpose(0, 1)[:, None] for x in ("k_cache", "v_cache"))  # [H, 1, N, D]
            q = state["q"][row:row + p1 - p0].float().view(p1 - p0, h, -1, d).permute(1, 2, 0, 3)  # [H, g, n, D]
            at = torch.arange(p0, p1, device="cuda")[:, None]
            mask = (token <= at) & ((token > at - case["window"]) | (token < case["sinks"]))
            o = _softmax_sum((q @ k.transpose(-1, -2)) * state["scale"], mask, v)
            out[row:row + p1 - p0] = o.permute(2, 0, 1, 3).reshape(p1 - p0, -1, d).to(out.dtype)
            row += p1 - p0
    return out


def _plain(state):
    op = state["case"]["op"]
    if op == "append8":
        return _append8(state)
    return {"out": _chunk(state) if op == "chunk" else _decode(state)}


# ---- the framework's calls --------------------------------------------------------------------------


def _own(s):
    import paged_kv_cache_126_gb300 as pa

    case = s["case"]
    op = case["op"]
    if op == "window":
        pa.pa_decode_window(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"], case["window"], s["scale"],
                            s["out"], sinks=case["sinks"])
    elif op == "chunk":
        pa.pa_prefill_window(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"], s["query_start"],
                             case["window"], s["scale"], s["out"], sinks=case["sinks"])
    elif op == "decode8":
        pa.pa_decode_q8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_tables"], s["context_lens"],
                        s["scale"], s["out"], window=case["window"], sinks=case["sinks"])
    else:
        pa.pa_cache_append_q8(s["k_new"], s["v_new"], s["block_tables"], s["context_lens"], s["k_cache"], s["v_cache"],
                              s["k_scale"], s["v_scale"], query_start=s["query_start"])
        pa.pa_cache_read_q8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["slots"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return {"out": s["out"]}


def run(state):
    if own:
        return _own(state)
    else:
        return _plain(state)


# ---- the definitions in 64 bits -----------------------------------------------------------------------


def _top_bits(x, bits=8):
    """x > 0 cut to its leading bits."""
    e = torch.floor(torch.log2(x)) - (bits - 1)
    return torch.floor(x * 2.0 ** -e) * 2.0 ** e


def _append64(case, s):
    """Frame by frame: the rate of the frame, halved while an element does not fit, and all its tokens coded in turn."""
    b, row = case["b"], 0
    steps = {x: s[x + "_scale"].double() for x in ("k", "v")}
    rows = {"k": [], "v": []}
    for i, (n, c) in enumerate(_lens(case)):
        for j in range((n - c) // b, -(-n // b)):
            f = int(s["block_tables"][i, j])
            fresh = range(max(n - c, j * b), min(n, (j + 1) * b))
            before = fresh[0] - j * b
            for x in ("k", "v"):
                new = s[x + "_new"][row:row + len(fresh)].double()  # [N, H, D]
                largest = new.abs().amax((0, 2)).clip(LEAST, MOST)
                codes = s[x + "_cache"][f, :, :before].double() - 128  # [H, before, D]
                if before:
                    halvings = torch.zeros_like(largest)
                    rate = _top_bits((1 / steps[x][f]) * (1 + 2.0 ** -20))  # the step is 1 / rate, rounded
                    while bool((largest * rate > 127).any()):
                        halvings += largest * rate > 127
                        rate = torch.where(largest * rate > 127, rate / 2, rate)
                    codes = torch.round(codes / 2.0 ** halvings[:, None, None])
                    steps[x][f] = steps[x][f] * 2.0 ** halvings
                else:
                    rate = _top_bits(127 / largest)
                    steps[x][f] = 1 / rate
                coded = torch.round(new.transpose(0, 1) * rate[:, None, None]).clip(-127, 127)
                rows[x].append((torch.cat([codes, coded], 1) * steps[x][f][:, None, None]).transpose(0, 1))
            row += len(fresh)
    return {"k": torch.cat(rows["k"]), "v": torch.cat(rows["v"]), "k_scale": steps["k"], "v_scale": steps["v"]}


def exact(case, seed):
    s = prepare(case, seed)
    op, h, d, b = case["op"], case["h"], case["d"], case["b"]
    if op == "append8":
        return _append64(case, s) if sum(len(_frames(case, n, c)) for n, c in _lens(case)) < 4000 else None
    group, row = case["hq"] // h, 0
    out = torch.zeros_like(s["q"], dtype=torch.float64)
    for i, (n, c) in enumerate(_lens(case)):
        seen = torch.tensor([j * b + o for j in _frames(case, n, c) for o in range(b) if j * b + o < n], device="cuda")
        frame, offset = s["block_tables"][i].long()[seen // b], seen % b
        for j in range(h):
            if op == "decode8":
                k, v = ((s[x + "_cache"][frame, j, offset].double() - 128) * s[x + "_scale"][frame, j].double()[:, None] for x in ("k", "v"))
            else:
                k, v = (s[x + "_cache"][frame, offset, j].double() for x in ("k", "v"))
            for t0 in range(0, c, 1024):
                at = torch.arange(n - c + t0, min(n, n - c + t0 + 1024), device="cuda")[:, None]
                hidden = seen > at
                if case["window"]:
                    hidden = hidden | ((seen <= at - case["window"]) & (seen >= case["sinks"]))
                live = ~hidden.all(0)
                for g in range(j * group, (j + 1) * group):
                    q = s["q"][row + t0:row + t0 + len(at), g].double()
                    a = torch.einsum("td,nd->tn", q, k[live]) * s["scale"]
                    a[hidden[:, live]] = -math.inf
                    out[row + t0:row + t0 + len(at), g] = torch.softmax(a, dim=-1) @ v[live]
        row += c
    return {"out": out}
