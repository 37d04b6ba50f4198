"""Measured cases of the key-value cache operators: quantizing keys and values
into a paged cache as they are written, reading them back, and the attention of
new tokens over the paged cache.

A cache holds K and V as pages [pages, kv_heads, page_size, head_dim].  With
4-bit and 8-bit codes a token's head_dim values are cut into groups of
`group_size`; each group stores an fp16 scale s and an fp16 bias b and stands
for q*s + b (the weight format of this package, one row per token and head).
With 16 bits the pages hold the values themselves.

`own` selects the package's operators; otherwise everything is computed from
elementary torch operations in binary32.
"""
import math
import random

import numpy as np
import torch

own = False

# the scratch memory of the attention call, which a program allocates and
# clears once and then passes to every step
WORKSPACE_BYTES = 64 << 20


# ---- cases -----------------------------------------------------------------------------
def listed():
    def attend(name, batch, longest, kv_heads, group, dim, bits, group_size, page, tokens, dtype,
               ragged, idle=0):
        return {"name": name, "op": "attend", "batch": batch, "longest": longest,
                "kv_heads": kv_heads, "group": group, "dim": dim, "bits": bits,
                "group_size": group_size, "page": page, "tokens": tokens, "dtype": dtype,
                "ragged": ragged, "idle": idle}

    def move(name, op, tokens, run, kv_heads, dim, bits, group_size, page, dtype):
        return {"name": name, "op": op, "tokens": tokens, "run": run, "kv_heads": kv_heads,
                "dim": dim, "bits": bits, "group_size": group_size, "page": page, "dtype": dtype}

    return [
        # the first steps of one conversation: nothing but latency (32 query and 8 key heads of
        # 128, the widths of the decode benchmark's [4096, 4096] and [1024, 4096] projections)
        attend("attend one short", 1, 37, 8, 4, 128, 8, 64, 16, 1, "f16", False),
        # one conversation with a whole book in its cache, 4-bit to hold it
        attend("attend one long", 1, 131072, 8, 4, 128, 4, 64, 64, 1, "bf16", False),
        # a server's ordinary step: sequences of every age
        attend("attend batch", 16, 4096, 8, 4, 128, 8, 64, 16, 1, "bf16", True),
        # a full server: the largest call
        attend("attend full", 64, 16384, 8, 4, 128, 8, 128, 64, 1, "bf16", True),
        # small heads, odd counts, pages that are no power of two, an idle slot in the batch
        attend("attend odd", 7, 777, 5, 7, 64, 4, 32, 48, 1, "f16", True, 1),
        # checking five drafted tokens at once (the speculative widths of the matmul benchmark)
        attend("attend draft", 8, 8192, 8, 8, 128, 8, 128, 32, 5, "bf16", True),
        # a cache that is kept in bfloat16
        attend("attend 16 bits", 16, 8192, 8, 4, 128, 16, 0, 16, 1, "bf16", True),
        # one key head of 256 shared by sixteen query heads
        attend("attend shared", 3, 20001, 1, 16, 256, 8, 64, 64, 1, "f16", True),
        # a decode step writes one token for each of 64 sequences
        move("write step", "write", 64, 1, 8, 128, 8, 64, 16, "f16"),
        # a prompt's tokens are written at once
        move("write prompt", "write", 8191, 512, 8, 128, 4, 64, 64, "bf16"),
        # a short shared prefix is read back
        move("read prefix", "read", 333, 333, 5, 64, 8, 32, 16, "f16"),
        # a long context is read back to attend to it in one product
        move("read long", "read", 65536, 8192, 8, 128, 4, 64, 64, "bf16"),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    dim = rng.choice([64, 128, 128, 256])
    bits = rng.choice([4, 8, 8, 16])
    case = {"kv_heads": rng.choice([1, 2, 4, 5, 8, 8, 16]), "dim": dim, "bits": bits,
            "group_size": 0 if bits == 16 else rng.choice([g for g in (32, 64, 128) if g <= dim]),
            "page": rng.choice([16, 16, 32, 48, 64, 128]), "dtype": rng.choice(["f16", "bf16"])}
    row = case["kv_heads"] * 2 * _row_bytes(case)
    if rng.random() < 0.7:
        case.update(op="attend", batch=spread(1, 64), longest=spread(1, 131072),
                    group=rng.choice([1, 2, 4, 5, 7, 8, 16]),
                    tokens=rng.choice([1, 1, 1, 2, 3, 5, 8]), ragged=rng.random() < 0.7)
        case["idle"] = 1 if case["batch"] > 3 and rng.random() < 0.3 else 0
        # no more cache than the largest listed case, and no more products
        most = 64 * 8192 * 8 * 2 * 132
        flops = 4 * dim * case["kv_heads"] * case["group"] * case["tokens"]
        tokens = min(most // row, 4 * dim * 32 * 5 * 8 * 8192 * 2 // flops)
        case["longest"] = max(1, min(case["longest"], tokens // case["batch"]))
        case["longest"] = max(case["longest"], case["tokens"])
    else:
        case.update(op=rng.choice(["write", "read"]))
        most = 65536 * 8 * 128 // (case["kv_heads"] * dim)
        case["tokens"] = spread(1, min(65536 if case["op"] == "read" else 16384, most))
        case["run"] = spread(1, case["tokens"])
    return case


def _row_bytes(case):
    """Bytes of one token's keys (or values) in one head of the cache."""
    d, bits = case["dim"], case["bits"]
    return d * 2 if bits == 16 else d * bits // 8 + d // case["group_size"] * 4


def _lengths(case):
    """Tokens in the cache of each sequence, the step's own among them: the same
    set for every seed, in another order."""
    n, top = case["batch"], case["longest"]
    rng = random.Random(n * 1000003 + top)
    got = [top] + [rng.randint(min(top, case["tokens"]), top) if case["ragged"] else top
                   for _ in range(n - 1)]
    for i in range(case["idle"]):
        got[-1 - i] = 0
    return got


def work(case):
    row = case["kv_heads"] * 2 * _row_bytes(case)
    wide = case["kv_heads"] * 2 * case["dim"] * 2
    if case["op"] != "attend":
        # the 16-bit rows once and the cache's rows once, and the slots
        return {"bytes": case["tokens"] * (row + wide + 8), "flops": 0}
    lengths = _lengths(case)
    heads = case["kv_heads"] * case["group"]
    seen = sum(max(0, n - case["tokens"] + 1 + i) for n in lengths for i in range(case["tokens"]))
    table = sum(-(-n // case["page"]) for n in lengths) + len(lengths)
    return {"bytes": sum(lengths) * row + 4 * table
            + 2 * len(lengths) * case["tokens"] * heads * case["dim"] * 2,
            "flops": 4 * case["dim"] * heads * seen}


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    heads, dim, page = case["kv_heads"], case["dim"], case["page"]
    dtype, bits = _DTYPES[case["dtype"]], case["bits"]
    state = {"case": case}

    def cache(pages, filled):
        shape = (pages, heads, page, dim)
        for name, make in (("k", _keys), ("v", _values)):
            if bits == 16:
                state[name] = (make(shape, gen, dtype) if filled
                               else torch.zeros(shape, dtype=dtype, device="cuda"), None, None)
            elif filled:
                state[name] = _pack(make(shape, gen, dtype), case["group_size"], bits)
            else:
                groups = shape[:3] + (dim // case["group_size"],)
                state[name] = (
                    torch.zeros(shape[:3] + (dim * bits // 32,), dtype=torch.int32, device="cuda"),
                    torch.zeros(groups, dtype=torch.float16, device="cuda"),
                    torch.zeros(groups, dtype=torch.float16, device="cuda"))

    if case["op"] == "attend":
        lengths = _lengths(case)
        rng.shuffle(lengths)
        need = [-(-n // page) for n in lengths]
        pages = sum(need) + 3
        order = list(range(pages))
        rng.shuffle(order)
        table = np.full((len(lengths), max(need)), -1, dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        cache(pages, True)
        state["table"] = torch.from_numpy(table).cuda()
        state["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        state["q"] = torch.randn((len(lengths), case["tokens"], heads * case["group"], dim),
                                 generator=gen, device="cuda").to(dtype)
        state["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
        return state

    # runs of consecutive tokens, each run starting a page of its own
    tokens, run_ = case["tokens"], case["run"]
    runs = -(-tokens // run_)
    per = -(-run_ // page)
    pages = runs * per + 3
    order = torch.randperm(pages, generator=gen, device="cuda")
    t = torch.arange(tokens, device="cuda")
    i = t % run_
    state["slots"] = order[(t // run_) * per + i // page] * page + i % page
    if case["op"] == "write":
        cache(pages, False)
        # keys and values of one fused projection, side by side in its rows
        both = torch.cat([_keys((tokens, heads, dim), gen, dtype).reshape(tokens, -1),
                          _values((tokens, heads, dim), gen, dtype).reshape(tokens, -1)], dim=1)
        state["new_k"] = both[:, :heads * dim].view(tokens, heads, dim)
        state["new_v"] = both[:, heads * dim:].view(tokens, heads, dim)
    else:
        cache(pages, True)
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


def _plain_write(state):
    case = state["case"]
    page = state["slots"] // case["page"], state["slots"] % case["page"]
    for name in ("k", "v"):
        new = state["new_" + name]
        parts = (new,) if case["bits"] == 16 else _pack(new, case["group_size"], case["bits"])
        [part.index_put_((page[0][:, None], torch.arange(case["kv_heads"], device="cuda")[None],
                          page[1][:, None]), value) for part, value in zip(state[name], parts)]
    return _plain_read(state)


def _plain_read(state):
    case = state["case"]
    page, at = state["slots"] // case["page"], state["slots"] % case["page"]

    def rows(parts):
        parts = [None if p is None else p[page, :, at] for p in parts]
        return _unpack(*parts, case["group_size"], case["bits"]).to(_DTYPES[case["dtype"]])

    return {"k": rows(state["k"]), "v": rows(state["v"])}


def _plain_attend(state):
    case, q = state["case"], state["q"]
    batch, tokens, heads, dim = q.shape
    kv_heads, group = case["kv_heads"], case["group"]
    table = state["table"].long().clamp(min=0)

    def rows(parts):  # [batch, kv_heads, positions, dim] of every page in the table
        parts = [None if p is None else p[table].transpose(1, 2).flatten(2, 3) for p in parts]
        return _unpack(*parts, case["group_size"], case["bits"])

    q = q.float().view(batch, tokens, kv_heads, group, dim).transpose(1, 2).flatten(2, 3)
    score = torch.matmul(q, rows(state["k"]).transpose(2, 3)) / math.sqrt(dim)
    positions = torch.arange(score.shape[-1], device="cuda")
    last = state["lengths"][:, None] - tokens + torch.arange(tokens, device="cuda")[None]
    sees = positions[None, None] <= last[:, :, None]
    sees = sees.repeat_interleave(group, dim=1)[:, None]
    score = score.masked_fill(~sees, -math.inf)
    most = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(most > -math.inf, most, torch.zeros_like(most)))
    total = p.sum(-1, keepdim=True)
    v = rows(state["v"])
    out = torch.matmul(p / torch.where(total > 0, total, torch.ones_like(total)), v)
    out = out.view(batch, kv_heads, tokens, group, dim).transpose(1, 2).flatten(2, 3)
    return {"out": out.to(state["q"].dtype)}


def run(state):
    case = state["case"]
    op, group_size, bits = case["op"], case["group_size"], case["bits"]
    if not own:
        return {"attend": _plain_attend, "write": _plain_write, "read": _plain_read}[op](state)
    import group_wise_affine_aq_amd as aq
    if op == "attend":
        return {"out": aq.aq_paged_attention(state["q"], *state["k"], *state["v"], state["table"],
                                             state["lengths"], group_size, bits,
                                             workspace=state["workspace"])}
    if op == "write":
        aq.aq_kv_append(state["new_k"], state["new_v"], state["slots"], *state["k"], *state["v"],
                        group_size, bits)
    k, v = aq.aq_kv_read(state["slots"], *state["k"], *state["v"], group_size, bits,
                         out_dtype=_DTYPES[case["dtype"]])
    return {"k": k, "v": v}


# ---- the definition in binary64 --------------------------------------------------------
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


def exact(case, seed):
    state = prepare(case, seed)
    page = case["page"]
    if case["op"] == "write":
        return {n: state["new_" + n].double() if case["bits"] == 16
                else _exact_grid(state["new_" + n], case["group_size"], case["bits"])
                for n in ("k", "v")}
    if case["op"] == "read":
        slots = state["slots"]
        return {n: _exact_rows([None if p is None else p[slots // page, :, slots % page]
                                for p in state[n]], case) for n in ("k", "v")}
    q = state["q"].double()
    out = torch.zeros_like(q)
    tokens, group = case["tokens"], case["group"]
    for i, n in enumerate(state["lengths"].tolist()):
        pages = state["table"][i, :-(-n // page)].long()
        for h in range(case["kv_heads"] if n else 0):
            k, v = (_exact_rows([None if p is None else p[pages, h].flatten(0, 1)[:n]
                                 for p in state[name]], case) for name in ("k", "v"))
            for t in range(tokens):
                sees = n - tokens + t + 1
                if sees > 0:
                    at = slice(h * group, (h + 1) * group)
                    w = torch.softmax(q[i, t, at] @ k[:sees].T * dim_scale(case), dim=-1)
                    out[i, t, at] = w @ v[:sees]
    return {"out": out}


def dim_scale(case):
    return case["dim"] ** -0.5
