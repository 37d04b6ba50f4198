"""Measured cases of the operators around the key-value cache: rotary positions
applied while keys and values are written into it, attention whose scores are
capped, biased by distance or masked (new tokens over the paged cache, and whole
prompts), the attention weight that every cached token gathers, and eviction of
the tokens that gathered least.

A cache holds K and V as pages [pages, kv_heads, page_size, head_dim].  With
4-bit and 8-bit codes a token's head_dim values are cut into groups of
`group_size`; each group stores an fp16 scale s and an fp16 bias b and stands
for q*s + b (the weight format of this package, one row per token and head).
With 16 bits the pages hold the values themselves.

`own` selects the package's operators; otherwise everything is computed from
elementary torch operations in binary32, angles of positions in binary64.
"""
import math
import random

import numpy as np
import torch

own = False

# the scratch memory of the attention calls, which a program allocates and
# clears once and then passes to every step
WORKSPACE_BYTES = 64 << 20


# ---- cases -----------------------------------------------------------------------------
def listed():
    def case(name, op, kv_heads, group, dim, dtype, **more):
        return {"name": name, "op": op, "kv_heads": kv_heads, "group": group, "dim": dim,
                "dtype": dtype, **more}

    def cache(bits, group_size, page):
        return {"bits": bits, "group_size": group_size, "page": page}

    def scores(softcap=0.0, slopes=False, window=0, first=False):
        return {"softcap": softcap, "slopes": slopes, "window": window, "first": first}

    return [
        # a decode step's new tokens of 64 sequences (32 query and 8 key heads of 128: the widths
        # of the decode benchmark's projections), positions anywhere in a long context
        case("rotate step", "rotate", 8, 4, 128, "f16", tokens=64, run=1, rotary=128,
             interleaved=False, farthest=32768, stretch=1.0, **cache(8, 64, 16)),
        # a prompt, its frequencies stretched for a context longer than was trained on
        case("rotate prompt", "rotate", 8, 4, 128, "bf16", tokens=8191, run=8191, rotary=128,
             interleaved=True, farthest=1000000, stretch=8.0, **cache(4, 64, 64)),
        # half of the head keeps its values, odd counts, pages that are no power of two
        case("rotate part", "rotate", 5, 7, 64, "f16", tokens=333, run=100, rotary=32,
             interleaved=False, farthest=4096, stretch=1.0, **cache(16, 0, 48)),
        # the first steps of one conversation, capped scores: nothing but latency
        case("attend capped short", "attend", 8, 4, 128, "f16", batch=1, longest=37, tokens=1,
             ragged=False, **cache(8, 64, 16), **scores(softcap=50.0)),
        # layers that look back 1024 tokens, sequences of every age
        case("attend window", "attend", 8, 4, 128, "bf16", batch=16, longest=8192, tokens=1,
             ragged=True, **cache(8, 64, 16), **scores(softcap=50.0, window=1024)),
        # a full server, scores biased by distance, documents that begin inside a sequence
        case("attend biased full", "attend", 8, 4, 128, "bf16", batch=64, longest=16384, tokens=1,
             ragged=True, **cache(4, 64, 64), **scores(slopes=True, first=True)),
        # one short prompt with small heads
        case("prompt short", "prompt", 4, 2, 64, "f16", batch=1, longest=61, past=0, ragged=False,
             prefix=False, **scores(softcap=30.0)),
        # several prompts in one call, some with a context before them, documents packed into
        # them, a prefix that all of a prompt's tokens see
        case("prompt packed", "prompt", 8, 4, 128, "f16", batch=6, longest=1501, past=777,
             ragged=True, prefix=True, **scores(slopes=True, first=True)),
        # a long prompt with capped scores: the largest call
        case("prompt long", "prompt", 8, 4, 128, "bf16", batch=1, longest=8192, past=0,
             ragged=False, prefix=False, **scores(softcap=50.0)),
        # after a decode step: what each cached token got of it
        case("weigh step", "weigh", 8, 4, 128, "bf16", batch=16, longest=4096, tokens=1,
             ragged=True, **cache(8, 64, 16), **scores()),
        # the last tokens of a long prompt ask what of it to keep
        case("weigh long", "weigh", 8, 4, 128, "bf16", batch=1, longest=131072, tokens=8,
             ragged=False, **cache(4, 64, 64), **scores()),
        # every sequence of a batch back to its budget
        case("evict batch", "evict", 8, 4, 128, "bf16", batch=24, longest=8192, keep=2048, sinks=4,
             recent=256, ragged=True, **cache(8, 64, 16)),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    dim = rng.choice([64, 128, 128, 256])
    case = {"op": rng.choice(["rotate", "attend", "attend", "prompt", "prompt", "weigh", "evict"]),
            "kv_heads": rng.choice([1, 2, 4, 5, 8, 8, 16]), "group": rng.choice([1, 2, 4, 5, 7, 8, 16]),
            "dim": dim, "dtype": rng.choice(["f16", "bf16"])}
    if case["op"] != "prompt":
        case["bits"] = rng.choice([4, 8, 8, 16])
        case["group_size"] = 0 if case["bits"] == 16 else rng.choice([g for g in (32, 64, 128) if g <= dim])
        case["page"] = rng.choice([16, 16, 32, 48, 64, 128])
        row = case["kv_heads"] * 2 * _row_bytes(case)
    if case["op"] in ("attend", "prompt", "weigh"):
        case.update(softcap=rng.choice([0.0, 0.0, 15.0, 50.0]), slopes=rng.random() < 0.3,
                    window=spread(16, 4096) if rng.random() < 0.3 else 0, first=rng.random() < 0.3,
                    ragged=rng.random() < 0.7)
    heads = case["kv_heads"] * case["group"]
    if case["op"] == "rotate":
        case.update(tokens=spread(1, max(1, 8191 * 40 * 128 // ((heads + 2 * case["kv_heads"]) * dim))),
                    rotary=dim // rng.choice([1, 1, 1, 2, 4]), interleaved=rng.random() < 0.5,
                    farthest=spread(100, 1000000), stretch=rng.choice([1.0, 4.0, 32.0]))
        case["run"] = spread(1, case["tokens"])
    elif case["op"] in ("attend", "weigh"):
        case.update(batch=spread(1, 64), longest=spread(1, 131072), tokens=rng.choice([1, 1, 2, 3, 8]))
        # no more cache than the largest listed case has in 8 bits, and no more products
        flops = 4 * dim * heads * case["tokens"]
        tokens = min(64 * 8192 * 8 * 2 * 132 // row, 4 * 128 * 32 * 64 * 16384 // flops)
        case["longest"] = max(case["tokens"], min(case["longest"], tokens // case["batch"]))
    elif case["op"] == "prompt":
        case.update(batch=spread(1, 16), longest=spread(1, 8192), prefix=rng.random() < 0.3,
                    past=spread(1, 8192) if rng.random() < 0.4 else 0)
        # every token against every token: no more than the long prompt, whose tokens see half
        most = 8192 * 8192 * 32 * 128 // (2 * case["batch"] * heads * dim)
        while case["longest"] * (case["longest"] + case["past"]) > most:
            case["longest"], case["past"] = case["longest"] * 7 // 8, case["past"] * 7 // 8
    else:
        case.update(batch=spread(1, 64), longest=spread(16, 65536), ragged=rng.random() < 0.7)
        case["longest"] = max(16, min(case["longest"], 24 * 8192 * 8 * 2 * 132 // row // case["batch"]))
        case["keep"] = spread(4, case["longest"])
        case["sinks"] = rng.randint(0, case["keep"] // 2)
        case["recent"] = rng.randint(0, case["keep"] - case["sinks"])
    return case


def _row_bytes(case):
    """Bytes of one token's keys (or values) in one head of the cache."""
    d, bits = case["dim"], case["bits"]
    return d * 2 if bits == 16 else d * bits // 8 + d // case["group_size"] * 4


def _lengths(case):
    """Tokens of each sequence (of a cache: the step's own among them): the same set for every
    seed, in another order."""
    n, top = case["batch"], case["longest"]
    rng = random.Random(n * 1000003 + top)
    least = min(top, case.get("tokens", 1))
    return [top] + [rng.randint(least, top) if case["ragged"] else top for _ in range(n - 1)]


def _sees(case, last, length, first, prefix):
    """How many of `length` tokens the token at position `last` sees, numpy arrays."""
    low = np.maximum(first, last - case["window"] + 1 if case["window"] else 0)
    high = np.maximum(np.minimum(np.maximum(last + 1, prefix), length), 0)
    return np.maximum(high - np.maximum(low, 0), 0)


def _first_of(case, n):
    """Where, within a sequence of n cached tokens, the newest token's document begins."""
    return n // 3 if case["first"] else 0


def _documents(case, n):
    """Where the document of each of a prompt's n tokens begins (its context included)."""
    if not case["first"]:
        return np.zeros(n, np.int64)
    rng = random.Random(n * 7919 + case["batch"])
    cuts = sorted({0, *(rng.randrange(n) for _ in range(rng.randint(1, 6)))})
    return np.repeat(cuts, np.diff(cuts + [n]))


def _prompts(case):
    """Per prompt: new tokens, tokens before them, tokens that all of it sees."""
    rng = random.Random(case["longest"] * 31 + case["batch"])
    got = []
    for n in _lengths(case):
        past = rng.randint(0, case["past"]) if case["ragged"] else case["past"]
        got.append((n, past, (past + n) // 4 if case["prefix"] else 0))
    return got


def work(case):
    dim, heads = case["dim"], case["kv_heads"] * case["group"]
    if case["op"] == "prompt":
        rows = keys = seen = 0
        for n, past, prefix in _prompts(case):
            first = _documents(case, past + n)[past:]
            seen += int(_sees(case, past + np.arange(n), past + n, first, prefix).sum())
            rows, keys = rows + n, keys + past + n
        return {"bytes": rows * heads * (4 * dim + 4) + keys * case["kv_heads"] * 4 * dim,
                "flops": 4 * dim * heads * seen}
    row = case["kv_heads"] * 2 * _row_bytes(case)
    if case["op"] == "rotate":
        # 16-bit rows of queries, keys and values read, rotated queries and the cache's rows written
        wide = (2 * heads + 2 * case["kv_heads"]) * dim * 2
        return {"bytes": case["tokens"] * (wide + row + 16), "flops": 0}
    lengths = _lengths(case)
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in lengths)
        return {"bytes": 4 * sum(lengths) + kept * (2 * row + 8), "flops": 0}
    seen = cached = 0
    for n in lengths:
        at = n - case["tokens"] + np.arange(case["tokens"])
        first = _first_of(case, n)
        seen += int(_sees(case, at, n, first, 0).sum())
        low = max(0, first, int(at[0]) - case["window"] + 1 if case["window"] else 0)
        cached += n - low
    table = sum(-(-n // case["page"]) for n in lengths) + len(lengths)
    rows = len(lengths) * case["tokens"] * heads
    if case["op"] == "attend":
        return {"bytes": cached * row + 4 * table + rows * (4 * dim + 4), "flops": 4 * dim * heads * seen}
    return {"bytes": cached * (row // 2 + 8) + 4 * table + rows * (2 * dim + 4),
            "flops": 2 * dim * heads * seen}


# ---- inputs ----------------------------------------------------------------------------
_DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _keys(shape, gen, dtype):
    """Keys as projections give them: a few channels far larger than the rest."""
    x = torch.randn(shape, generator=gen, device="cuda")
    loud = torch.ones(shape[-1], device="cuda")
    loud[::29] = 6.0
    return (x * loud).to(dtype)


def _values(shape, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _make_cache(case, state, gen, pages, filled):
    dim, bits, dtype = case["dim"], case["bits"], _DTYPES[case["dtype"]]
    shape = (pages, case["kv_heads"], case["page"], dim)
    for name, make in (("k", _keys), ("v", _values)):
        if bits == 16:
            state[name] = (make(shape, gen, dtype) if filled
                           else torch.zeros(shape, dtype=dtype, device="cuda"), None, None)
        elif filled:
            state[name] = _pack(make(shape, gen, dtype), case["group_size"], bits)
        else:
            groups = shape[:3] + (dim // case["group_size"],)
            state[name] = (torch.zeros(shape[:3] + (dim * bits // 32,), dtype=torch.int32, device="cuda"),
                           torch.zeros(groups, dtype=torch.float16, device="cuda"),
                           torch.zeros(groups, dtype=torch.float16, device="cuda"))


def _tables(need, order):
    """Page tables [sequences, max(need)] from a list of page numbers."""
    table = np.full((len(need), max(need)), -1, dtype=np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table).cuda()


def _slopes(case):
    heads = case["kv_heads"] * case["group"]
    if not case["slopes"]:
        return None
    return torch.exp2(-8.0 * torch.arange(1, heads + 1, device="cuda").float() / heads)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    heads, dim, dtype = case["kv_heads"], case["dim"], _DTYPES[case["dtype"]]
    state = {"case": case}
    return {"rotate": _prepare_rotate, "prompt": _prepare_prompt, "evict": _prepare_evict,
            "attend": _prepare_attend, "weigh": _prepare_attend}[case["op"]](
        case, state, gen, rng, heads, dim, dtype)


def _prepare_rotate(case, state, gen, rng, heads, dim, dtype):
    # runs of consecutive tokens, each run starting a page of its own at a position of its own
    tokens, run_, page = case["tokens"], case["run"], case["page"]
    runs = -(-tokens // run_)
    per = -(-run_ // page)
    pages = runs * per + 3
    order = torch.randperm(pages, generator=gen, device="cuda")
    t = torch.arange(tokens, device="cuda")
    i = t % run_
    state["slots"] = order[(t // run_) * per + i // page] * page + i % page
    start = torch.randint(0, max(1, case["farthest"] - run_), (runs,), generator=gen, device="cuda")
    state["positions"] = (start[t // run_] + i).to(torch.int32)
    # the frequencies and the factor that a model holds; stretched ones for longer contexts
    half = case["rotary"] // 2
    freqs = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    state["freqs"] = (freqs / case["stretch"]).float()
    state["factor"] = 0.1 * math.log(case["stretch"]) + 1.0
    _make_cache(case, state, gen, pages, False)
    # queries, keys and values of one fused projection, side by side in its rows
    every = torch.cat([_values((tokens, heads * case["group"] * dim), gen, dtype),
                       _keys((tokens, heads, dim), gen, dtype).reshape(tokens, -1),
                       _values((tokens, heads * dim), gen, dtype)], dim=1)
    q, k, v = every.split([heads * case["group"] * dim, heads * dim, heads * dim], dim=1)
    state["q"], state["new_k"], state["new_v"] = (x.unflatten(1, (-1, dim)) for x in (q, k, v))
    return state


def _prepare_prompt(case, state, gen, rng, heads, dim, dtype):
    prompts = _prompts(case)
    rng.shuffle(prompts)
    rows, keys = (np.cumsum([0] + x).astype(np.int32)
                  for x in ([n for n, _, _ in prompts], [n + past for n, past, _ in prompts]))
    state["q_starts"], state["k_starts"] = torch.from_numpy(rows).cuda(), torch.from_numpy(keys).cuda()
    state["longest"] = max(n for n, _, _ in prompts), max(n + past for n, past, _ in prompts)
    state["q"] = _values((int(rows[-1]), heads * case["group"], dim), gen, dtype)
    # keys and values side by side in the rows of one projection
    both = torch.cat([_keys((int(keys[-1]), heads, dim), gen, dtype).flatten(1),
                      _values((int(keys[-1]), heads * dim), gen, dtype)], dim=1)
    state["k"], state["v"] = (x.unflatten(1, (heads, dim)) for x in both.split(heads * dim, dim=1))
    state["slopes"] = _slopes(case)
    state["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    state["prefix"] = state["first"] = None
    if case["prefix"]:
        state["prefix"] = torch.tensor([p for _, _, p in prompts], dtype=torch.int32, device="cuda")
    if case["first"]:
        first = np.concatenate([_documents(case, n + past)[past:] for n, past, _ in prompts])
        state["first"] = torch.from_numpy(first.astype(np.int32)).cuda()
    return state


def _prepare_attend(case, state, gen, rng, heads, dim, dtype):
    lengths, page = _lengths(case), case["page"]
    rng.shuffle(lengths)
    need = [-(-n // page) for n in lengths]
    order = list(range(sum(need) + 3))
    rng.shuffle(order)
    _make_cache(case, state, gen, len(order), True)
    state["table"] = _tables(need, order)
    state["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    state["q"] = torch.randn((len(lengths), case["tokens"], heads * case["group"], dim),
                             generator=gen, device="cuda").to(dtype)
    state["slopes"] = _slopes(case)
    state["first"] = None
    if case["first"]:
        state["first"] = torch.tensor([_first_of(case, n) for n in lengths], dtype=torch.int32,
                                      device="cuda")
    if case["op"] == "attend":
        state["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    else:
        # what the step's attention left: the logarithm of each row's sum of weights
        score, sees = _paged_scores(state)
        lse = torch.logsumexp(score.masked_fill_(~sees, -math.inf), dim=-1)
        state["lse"] = _rows_first(lse.unsqueeze(-1), case).squeeze(-1).contiguous()
        # and what earlier steps gathered
        state["before"] = torch.rand((len(lengths), max(need) * page), generator=gen, device="cuda") * 0.01
    return state


def _prepare_evict(case, state, gen, rng, heads, dim, dtype):
    lengths, page = _lengths(case), case["page"]
    rng.shuffle(lengths)
    need = [-(-n // page) for n in lengths]
    new = [-(-min(n, case["keep"]) // page) for n in lengths]
    order = list(range(sum(need) + sum(new) + 3))
    rng.shuffle(order)
    _make_cache(case, state, gen, len(order), True)
    state["table"], state["new_table"] = _tables(need, order), _tables(new, order[sum(need):])
    state["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    # weights gathered over many steps: a few tokens have most, many have equal small ones
    w = torch.exp(3 * torch.randn((len(lengths), max(need) * page), generator=gen, device="cuda"))
    state["weights"] = torch.round(w * 256) / 256
    # where the kept tokens' rows lie, to read them
    t = torch.arange(max(new) * page, device="cuda")
    slots = state["new_table"].long()[:, t // page] * page + t % page
    kept = torch.minimum(state["lengths"], torch.tensor(case["keep"], device="cuda"))
    state["new_slots"] = slots[t[None] < kept[:, None]]
    return state


# ---- plain forms, in binary32 ----------------------------------------------------------
def _half_step(h, up):
    """The neighbouring binary16 of a scale >= 0, one step up or down."""
    return (h.view(torch.int16) + (1 if up else -1)).clamp(0, 0x7BFF).to(torch.int16).view(torch.float16)


def _pack(x, group_size, bits):
    """Rows of the last axis -> (int32 words, fp16 scales, fp16 biases)."""
    top = float((1 << bits) - 1)
    x = x.float().unflatten(-1, (-1, group_size))
    lo, hi = x.amin(-1), x.amax(-1)
    # the bias is the largest binary16 that is no larger than any member
    b = lo.half()
    over = b.float() > lo
    raw = b.view(torch.int16)
    down = torch.where(b == 0, torch.full_like(raw, -0x7FFF), torch.where(raw < 0, raw + 1, raw - 1))
    b = torch.where(over, down.view(torch.float16), b) + 0.0
    # the scale is the smallest binary16 whose grid reaches the largest member
    s = ((hi - b.float()) / top).half()
    s = torch.where(b.float() + top * s.float() < hi, _half_step(s, True), s)
    less = _half_step(s, False)
    s = torch.where((s > 0) & (b.float() + top * less.float() >= hi), less, s)
    s = torch.where(b.float() >= hi, torch.zeros_like(s), s)
    step = s.float().unsqueeze(-1)
    q = torch.round((x - b.float().unsqueeze(-1)) / torch.where(step > 0, step, torch.ones_like(step)))
    q = torch.where(step > 0, q.clamp(0, top), torch.zeros_like(q)).to(torch.uint8).flatten(-2)
    if bits == 4:
        q = q[..., 0::2] | (q[..., 1::2] << 4)
    return q.contiguous().view(torch.int32), s, b


def _unpack(words, scales, biases, group_size, bits):
    """The values that packed rows stand for, in binary32."""
    if bits == 16:
        return words.float()
    q = words.contiguous().view(torch.uint8)
    if bits == 4:
        q = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2)
    q = q.float().unflatten(-1, (-1, group_size))
    return (q * scales.float().unsqueeze(-1) + biases.float().unsqueeze(-1)).flatten(-2)


def _read(state, slots):
    """Rows of the cache in the case's 16-bit type."""
    case = state["case"]
    page, at = slots // case["page"], slots % case["page"]
    got = {}
    for name in ("k", "v"):
        parts = [None if p is None else p[page, :, at] for p in state[name]]
        got[name] = _unpack(*parts, case["group_size"], case["bits"]).to(_DTYPES[case["dtype"]])
    return got


def _turn(x, cos, sin, interleaved):
    """Pairs of the first values of each head turned by the token's angles."""
    half = cos.shape[-1]
    part, rest = x[..., :2 * half].float(), x[..., 2 * half:]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :half], part[..., half:])
    cos, sin = cos[:, None], sin[:, None]
    a, b = a * cos - b * sin, b * cos + a * sin
    part = torch.stack((a, b), dim=-1).flatten(-2) if interleaved else torch.cat((a, b), dim=-1)
    return torch.cat((part.to(x.dtype), rest), dim=-1)


def _plain_rotate(state):
    case = state["case"]
    angles = state["positions"].double()[:, None] * state["freqs"].double()
    cos, sin = ((f(angles) * state["factor"]).float() for f in (torch.cos, torch.sin))
    q, k = (_turn(state[n], cos, sin, case["interleaved"]) for n in ("q", "new_k"))
    page, at = state["slots"] // case["page"], state["slots"] % case["page"]
    where = (page[:, None], torch.arange(case["kv_heads"], device="cuda")[None], at[:, None])
    for name, new in (("k", k), ("v", state["new_v"])):
        parts = (new,) if case["bits"] == 16 else _pack(new, case["group_size"], case["bits"])
        for part, value in zip(state[name], parts):
            part.index_put_(where, value)
    return {"q": q, **_cache_rows(state, state["slots"])}


def _cache_rows(state, slots):
    """The written rows: of a 16-bit cache the cache itself, else what its codes stand for."""
    return {n: state[n][0] for n in ("k", "v")} if state["case"]["bits"] == 16 else _read(state, slots)


def _adjust(score, case, slopes, distance):
    """Scaled scores -> capped and biased by the distance of their tokens."""
    if case["softcap"]:
        score = case["softcap"] * torch.tanh(score / case["softcap"])
    if slopes is not None:
        score = score - slopes * distance.abs().float()
    return score


def _softmax_rows(score, sees, v):
    """(weighted sum of v, logarithm of the sum of weights) in the rows that see anything."""
    score = score.masked_fill(~sees, -math.inf)
    most = score.amax(-1, keepdim=True)
    most = torch.where(most > -math.inf, most, torch.zeros_like(most))
    p = torch.exp(score - most)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p / torch.where(total > 0, total, torch.ones_like(total)), v)
    return out, most + torch.log(total)


def _rows_first(x, case):
    """[batch, kv_heads, tokens * group, n] -> [batch, tokens, kv_heads * group, n]"""
    return x.unflatten(2, (-1, case["group"])).transpose(1, 2).flatten(2, 3)


def _paged_rows(parts, state):
    """[batch, kv_heads, positions, dim] of every page in the table."""
    case = state["case"]
    table = state["table"].long().clamp(min=0)
    parts = [None if p is None else p[table].transpose(1, 2).flatten(2, 3) for p in parts]
    return _unpack(*parts, case["group_size"], case["bits"])


def _paged_scores(state):
    """Scores of the new tokens against every position of the table, and which count."""
    case, q = state["case"], state["q"]
    batch, tokens, heads, dim = q.shape
    kv_heads, group = case["kv_heads"], case["group"]
    q = q.float().view(batch, tokens, kv_heads, group, dim).transpose(1, 2).flatten(2, 3)
    score = torch.matmul(q, _paged_rows(state["k"], state).transpose(2, 3)) / math.sqrt(dim)
    t = torch.arange(score.shape[-1], device="cuda")
    last = state["lengths"][:, None] - tokens + torch.arange(tokens, device="cuda")[None]
    distance = (last[:, :, None] - t).repeat_interleave(group, dim=1)[:, None]
    sees = distance >= 0
    if case["window"]:
        sees &= distance < case["window"]
    if state["first"] is not None:
        sees &= t >= state["first"][:, None, None, None]
    slopes = state["slopes"]
    if slopes is not None:
        slopes = slopes.view(kv_heads, 1, group).expand(-1, tokens, -1).reshape(kv_heads, -1, 1)
    return _adjust(score, case, slopes, distance), sees


def _plain_attend(state):
    case = state["case"]
    score, sees = _paged_scores(state)
    out, lse = _softmax_rows(score, sees, _paged_rows(state["v"], state))
    return {"out": _rows_first(out, case).to(state["q"].dtype), "lse": _rows_first(lse, case).squeeze(-1)}


def _plain_weigh(state):
    case = state["case"]
    score, sees = _paged_scores(state)
    lse = state["lse"].unflatten(2, (case["kv_heads"], -1)).transpose(1, 2).flatten(2, 3).unsqueeze(-1)
    p = torch.where(sees, torch.exp(score - lse), torch.zeros_like(score))
    return {"weights": state["before"] + p.sum(dim=(1, 2))}


def _plain_prompt(state):
    case = state["case"]
    kv_heads, group, dim = case["kv_heads"], case["group"], case["dim"]
    rows, keys = state["longest"]

    def padded(x, starts, most):  # [batch, heads, most, dim] and which are there
        at = torch.arange(most, device="cuda")[None] + starts[:-1, None]
        return x[at.clamp(max=x.shape[0] - 1)].transpose(1, 2).float(), at < starts[1:, None]

    q, on = padded(state["q"], state["q_starts"], rows)
    k, there = padded(state["k"], state["k_starts"], keys)
    v, _ = padded(state["v"], state["k_starts"], keys)
    q = q.unflatten(1, (kv_heads, group))
    score = torch.matmul(q, k.transpose(2, 3).unsqueeze(2)) / math.sqrt(dim)
    past = torch.diff(state["k_starts"]) - torch.diff(state["q_starts"])
    t = torch.arange(keys, device="cuda")
    distance = (past[:, None] + torch.arange(rows, device="cuda")[None])[:, :, None] - t
    sees = distance >= 0
    if state["prefix"] is not None:
        sees |= t < state["prefix"][:, None, None]
    if case["window"]:
        sees &= distance < case["window"]
    if state["first"] is not None:
        first, _ = padded(state["first"][:, None, None], state["q_starts"], rows)
        sees &= t >= first[:, 0]
    sees &= there[:, None]
    slopes = state["slopes"]
    if slopes is not None:
        slopes = slopes.view(kv_heads, group, 1, 1)
    score = _adjust(score, case, slopes, distance[:, None, None])
    out, lse = _softmax_rows(score, sees[:, None, None], v.unsqueeze(2))
    out, lse = (x.flatten(1, 2).transpose(1, 2)[on] for x in (out, lse))
    return {"out": out.to(state["q"].dtype), "lse": lse.squeeze(-1)}


def _plain_evict(state):
    case = state["case"]
    keep, page = case["keep"], case["page"]
    weights, lengths = state["weights"], state["lengths"].long()[:, None]
    t = torch.arange(weights.shape[1], device="cuda")[None]
    # the first and the last tokens stay, then the largest weights, equal ones from the lowest
    # place on; places past the sequence come last
    rank = torch.where((t < case["sinks"]) | (t >= lengths - case["recent"]), math.inf, weights)
    rank = torch.where(t < lengths, rank, -math.inf)
    best = torch.argsort(rank, dim=1, descending=True, stable=True)[:, :keep]
    best, _ = torch.sort(torch.where(best < lengths, best, 1 << 30), dim=1)
    kept = torch.nn.functional.pad(best, (0, keep - best.shape[1]), value=1 << 30)
    on = kept < lengths
    kept = torch.where(on, kept, -1)
    old = torch.gather(state["table"].long(), 1, kept.clamp(min=0) // page) * page + kept.clamp(min=0) % page
    old, new = old[on], state["new_slots"]
    heads = torch.arange(case["kv_heads"], device="cuda")[None]
    for part in (*state["k"], *state["v"]):
        if part is not None:
            rows = part[(old // page)[:, None], heads, (old % page)[:, None]]
            part.index_put_(((new // page)[:, None], heads, (new % page)[:, None]), rows)
    got = torch.where(on, torch.gather(weights, 1, kept.clamp(min=0)), torch.zeros((), device="cuda"))
    return {"kept": kept.to(torch.int32), "lengths": torch.clamp(state["lengths"], max=keep),
            "weights": got, **_cache_rows(state, new)}


def run(state):
    case = state["case"]
    if not own:
        return {"rotate": _plain_rotate, "attend": _plain_attend, "prompt": _plain_prompt,
                "weigh": _plain_weigh, "evict": _plain_evict}[case["op"]](state)
    import group_wise_affine_aq_amd as aq
    dtype = _DTYPES[case["dtype"]]
    if case["op"] == "prompt":
        out, lse = aq.aq_prompt_attention(
            state["q"], state["k"], state["v"], state["q_starts"], state["k_starts"],
            softcap=case["softcap"], slopes=state["slopes"], window=case["window"],
            first=state["first"], prefix=state["prefix"], return_lse=True,
            workspace=state["workspace"])
        return {"out": out, "lse": lse}
    packing = (case["group_size"], case["bits"])
    if case["op"] == "attend":
        out, lse = aq.aq_paged_attention_masked(
            state["q"], *state["k"], *state["v"], state["table"], state["lengths"], *packing,
            softcap=case["softcap"], slopes=state["slopes"], window=case["window"],
            first=state["first"], return_lse=True, workspace=state["workspace"])
        return {"out": out, "lse": lse}
    if case["op"] == "weigh":
        weights = state["before"].clone()
        aq.aq_kv_weigh(state["q"], state["lse"], *state["k"], *state["v"], state["table"],
                       state["lengths"], weights, *packing, softcap=case["softcap"],
                       slopes=state["slopes"], window=case["window"], first=state["first"])
        return {"weights": weights}

    def rows(slots):
        if case["bits"] == 16:
            return {"k": state["k"][0], "v": state["v"][0]}
        k, v = aq.aq_kv_read(slots, *state["k"], *state["v"], *packing, out_dtype=dtype)
        return {"k": k, "v": v}

    if case["op"] == "rotate":
        q = aq.aq_rope_append(state["q"], state["new_k"], state["new_v"], state["positions"],
                              state["freqs"], state["slots"], *state["k"], *state["v"], *packing,
                              interleaved=case["interleaved"], factor=state["factor"])
        return {"q": q, **rows(state["slots"])}
    kept, lengths, weights = aq.aq_kv_evict(
        state["weights"], state["lengths"], state["table"], state["new_table"], *state["k"],
        *state["v"], *packing, keep=case["keep"], sinks=case["sinks"], recent=case["recent"])
    return {"kept": kept, "lengths": lengths, "weights": weights, **rows(state["new_slots"])}


# ---- the definitions in binary64 -------------------------------------------------------
def _exact_grid(x, group_size, bits):
    """What quantized rows stand for: exact comparisons against every binary16."""
    every = torch.arange(0, 0x7C00, dtype=torch.int16, device=x.device).view(torch.float16).double()
    signed = torch.cat([-every.flip(0)[:-1], every])
    levels = (1 << bits) - 1
    g = x.double().reshape(x.shape[:-1] + (-1, group_size))
    lo, hi = g.min(-1).values, g.max(-1).values
    b = signed[torch.searchsorted(signed, lo, right=True) - 1]
    s = every[torch.searchsorted(every * levels, hi - b)]
    b, s = b[..., None], s[..., None]
    n = torch.where(s > 0, torch.round((g - b) / s.clamp(min=2.0 ** -24)), torch.zeros_like(g))
    return (n.clamp(0, levels) * s + b).reshape(x.shape)


def _exact_rows(parts, case):
    words, scales, biases = parts
    if case["bits"] == 16:
        return words.double()
    bits, g = case["bits"], case["group_size"]
    shifts = torch.arange(0, 32, bits, device=words.device)
    n = ((words.long()[..., None] >> shifts) & ((1 << bits) - 1)).double()
    n = n.reshape(scales.shape + (g,))
    return (n * scales.double()[..., None] + biases.double()[..., None]).reshape(words.shape[:-1] + (-1,))


def _exact_rotated(x, angles, case, factor):
    """In complex numbers; rounded once to the rows' type."""
    half, z = case["rotary"] // 2, torch.polar(torch.full_like(angles, factor), angles)[:, None]
    y = x.double()
    pairs = (y[..., :2 * half].unflatten(-1, (half, 2)) if case["interleaved"]
             else y[..., :2 * half].unflatten(-1, (2, half)).transpose(-1, -2))
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    y = y.clone()
    y[..., :2 * half] = (turned if case["interleaved"] else turned.transpose(-1, -2)).flatten(-2)
    return y


def _exact_cache(state, new, slots):
    """A 16-bit cache after rows were written, or the written rows of a packed one."""
    case, got = state["case"], {}
    for n in ("k", "v"):
        if case["bits"] == 16:
            got[n] = state[n][0].double()
            got[n][slots // case["page"], :, slots % case["page"]] = new[n].double()
        else:
            got[n] = new[n].double()
    return got


def _exact_attention(q, k, v, case, at, low, high, slopes):
    """(rows, logarithms) of one head's queries [n, dim]; token i is at position at[i] and sees
    the tokens low[i] <= t < high[i]."""
    t = torch.arange(k.shape[0], device=k.device)
    s = q @ k.T * case["dim"] ** -0.5
    if case["softcap"]:
        s = torch.tanh(s / case["softcap"]) * case["softcap"]
    if slopes is not None:
        s = s - slopes[:, None].double() * (at[:, None] - t).abs()
    s = torch.where((t >= low[:, None]) & (t < high[:, None]), s, -math.inf)
    lse = torch.logsumexp(s, dim=1)
    return torch.nan_to_num(torch.exp(s - lse[:, None])), lse


def _bounds(case, at, length, first, prefix):
    low = first.clone()
    if case["window"]:
        low = torch.maximum(low, at - case["window"] + 1)
    return low, torch.clamp(torch.maximum(at + 1, torch.full_like(at, prefix)), max=length)


def _exact_paged(case, state):
    q, tokens, group, page = state["q"].double(), case["tokens"], case["group"], case["page"]
    out, lse = torch.zeros_like(q), torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    weights = state["before"].double() if case["op"] == "weigh" else None
    for b, n in enumerate(state["lengths"].tolist()):
        pages = state["table"][b, :-(-n // page)].long()
        at = n - tokens + torch.arange(tokens, device="cuda")
        first = torch.full_like(at, _first_of(case, n))
        low, high = (x.repeat_interleave(group) for x in _bounds(case, at, n, first, 0))
        for h in range(case["kv_heads"]):
            heads = slice(h * group, (h + 1) * group)
            k, v = (_exact_rows([None if p is None else p[pages, h].flatten(0, 1)[:n]
                                 for p in state[name]], case) for name in ("k", "v"))
            slopes = None if state["slopes"] is None else state["slopes"][heads].repeat(tokens)
            p, l = _exact_attention(q[b, :, heads].reshape(-1, q.shape[-1]), k, v, case,
                                    at.repeat_interleave(group), low, high, slopes)
            if weights is None:
                out[b, :, heads] = (p @ v).view(tokens, group, -1)
                lse[b, :, heads] = l.view(tokens, group)
            else:
                # against the logarithms that the call is given
                given = state["lse"][b, :, heads].reshape(-1).double()
                p = p * torch.exp(torch.where(l > -math.inf, l - given, 0.0))[:, None]
                weights[b, :n] += p.sum(0)
    return {"out": out, "lse": lse} if weights is None else {"weights": weights}


def _exact_prompt(case, state):
    q, k, v = (state[n].double() for n in ("q", "k", "v"))
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    rows, keys = state["q_starts"].tolist(), state["k_starts"].tolist()
    for b in range(len(rows) - 1):
        mine, length = slice(rows[b], rows[b + 1]), keys[b + 1] - keys[b]
        n = rows[b + 1] - rows[b]
        at = length - n + torch.arange(n, device="cuda")
        first = torch.zeros_like(at) if state["first"] is None else state["first"][mine].long()
        prefix = 0 if state["prefix"] is None else int(state["prefix"][b])
        low, high = _bounds(case, at, length, first, prefix)
        for h in range(q.shape[1]):
            kh, vh = (x[keys[b]:keys[b + 1], h // case["group"]] for x in (k, v))
            slopes = None if state["slopes"] is None else state["slopes"][h].expand(n)
            p, lse[mine, h] = _exact_attention(q[mine, h], kh, vh, case, at, low, high, slopes)
            out[mine, h] = p @ vh
    return {"out": out, "lse": lse}


def _exact_evict(case, state):
    page, keep = case["page"], case["keep"]
    batch = len(state["lengths"])
    kept = np.full((batch, keep), -1)
    got = np.zeros((batch, keep))
    weights, table = state["weights"].cpu().numpy(), state["table"].cpu().numpy()
    old = []
    for b, n in enumerate(state["lengths"].tolist()):
        stay = list(range(n))
        if n > keep:
            sinks, recent = range(case["sinks"]), range(n - case["recent"], n)
            between = np.arange(case["sinks"], n - case["recent"])
            order = np.lexsort((between, -weights[b, between].astype(np.float64)))
            stay = sorted([*sinks, *recent, *between[order[:keep - case["sinks"] - case["recent"]]].tolist()])
        kept[b, :len(stay)] = stay
        got[b, :len(stay)] = weights[b, stay]
        old += [int(table[b, t // page]) * page + t % page for t in stay]
    old = torch.tensor(old, device="cuda")
    new = {n: _exact_rows([None if p is None else p[old // page, :, old % page] for p in state[n]], case)
           for n in ("k", "v")}
    return {"kept": torch.from_numpy(kept), "lengths": torch.clamp(state["lengths"], max=keep),
            "weights": torch.from_numpy(got), **_exact_cache(state, new, state["new_slots"])}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] in ("attend", "weigh"):
        return _exact_paged(case, state)
    if case["op"] == "prompt":
        return _exact_prompt(case, state)
    if case["op"] == "evict":
        return _exact_evict(case, state)
    angles = state["positions"].double()[:, None] * state["freqs"].double()
    q = _exact_rotated(state["q"], angles, case, state["factor"])
    k = _exact_rotated(state["new_k"], angles, case, state["factor"]).to(_DTYPES[case["dtype"]])
    new = {"k": k, "v": state["new_v"]}
    if case["bits"] != 16:
        new = {n: _exact_grid(x, case["group_size"], case["bits"]) for n, x in new.items()}
    return {"q": q, **_exact_cache(state, new, state["slots"])}
