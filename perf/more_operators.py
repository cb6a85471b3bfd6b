"""Timed cases of serving long streams in bounded memory over the paged cache.

Each case is one call of one of these operators:
  stream    attention of every row's newest tokens -- one, a chunk, a whole prompt -- over its paged cache, each token seeing the
            `window` most recent tokens and the row's `first` ones; the cache in bf16, 8 bits (FP8) or 4 bits (NVFP4)
  release   gives back the pages that every later token's window has left behind

`run` computes them in elementary torch operations (32-bit, rounded once at the end), or, where `own` is true, by the
framework's entry points.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one user's next token in a windowed layer: latency
        {"name": "stream-bf16-token", "op": "stream", "fmt": "bf16", "batch": 1, "single": 1, "new_lo": 1, "new_hi": 1,
         "hq": 32, "hkv": 8, "dim": 128, "page": 16, "lo": 4000, "hi": 4000, "window": 1024, "first": 4},
        # single tokens at concurrency, long and short contexts together
        {"name": "stream-bf16-decode", "op": "stream", "fmt": "bf16", "batch": 32, "single": 32, "new_lo": 1, "new_hi": 1,
         "hq": 64, "hkv": 8, "dim": 128, "page": 32, "lo": 128, "hi": 16384, "window": 4096, "first": 128},
        # a whole prompt in a layer without a window
        {"name": "stream-bf16-prompt", "op": "stream", "fmt": "bf16", "batch": 1, "single": 0, "new_lo": 8192,
         "new_hi": 8192, "hq": 32, "hkv": 8, "dim": 128, "page": 16, "lo": 8192, "hi": 8192, "window": 0, "first": 0},
        # chunks of several long prompts in a windowed layer
        {"name": "stream-bf16-chunks", "op": "stream", "fmt": "bf16", "batch": 6, "single": 0, "new_lo": 500,
         "new_hi": 2048, "hq": 64, "hkv": 8, "dim": 128, "page": 32, "lo": 2048, "hi": 32768, "window": 4096,
         "first": 64},
        # a serving step of single tokens and a few chunks, small heads in odd groups, a short window
        {"name": "stream-bf16-mixed", "op": "stream", "fmt": "bf16", "batch": 24, "single": 20, "new_lo": 97,
         "new_hi": 701, "hq": 14, "hkv": 2, "dim": 64, "page": 64, "lo": 130, "hi": 9001, "window": 512, "first": 17},
        # short chunks with wide heads in a sliding-window layer
        {"name": "stream-bf16-wide", "op": "stream", "fmt": "bf16", "batch": 16, "single": 0, "new_lo": 33, "new_hi": 33,
         "hq": 16, "hkv": 4, "dim": 256, "page": 32, "lo": 2048, "hi": 32768, "window": 4096, "first": 4},
        # single tokens over an 8-bit cache, no window
        {"name": "stream-fp8-decode", "op": "stream", "fmt": "fp8", "batch": 32, "single": 32, "new_lo": 1, "new_hi": 1,
         "hq": 64, "hkv": 8, "dim": 128, "page": 32, "lo": 128, "hi": 16384, "window": 0, "first": 0},
        # two prompts' next chunks over an 8-bit cache
        {"name": "stream-fp8-chunks", "op": "stream", "fmt": "fp8", "batch": 2, "single": 0, "new_lo": 2048,
         "new_hi": 2048, "hq": 32, "hkv": 8, "dim": 128, "page": 16, "lo": 8192, "hi": 16384, "window": 0, "first": 0},
        # single tokens at high concurrency over a 4-bit cache, a wide window
        {"name": "stream-nvfp4-decode", "op": "stream", "fmt": "nvfp4", "batch": 64, "single": 64, "new_lo": 1,
         "new_hi": 1, "hq": 32, "hkv": 8, "dim": 128, "page": 32, "lo": 512, "hi": 32768, "window": 8192, "first": 4},
        # ragged chunks over a 4-bit cache in a windowed layer
        {"name": "stream-nvfp4-chunks", "op": "stream", "fmt": "nvfp4", "batch": 4, "single": 0, "new_lo": 300,
         "new_hi": 1500, "hq": 64, "hkv": 8, "dim": 128, "page": 32, "lo": 4096, "hi": 16384, "window": 2048,
         "first": 64},
        # after a step of single tokens: some rows' windows have passed a page
        {"name": "release-decode", "op": "release", "batch": 512, "page": 16, "new": 1, "lo": 16, "hi": 32768,
         "window": 4096, "first": 64, "ended": 0},
        # after a step of long chunks: many pages of every row, and rows that have ended
        {"name": "release-prompts", "op": "release", "batch": 64, "page": 16, "new": 2048, "lo": 1000, "hi": 131072,
         "window": 4096, "first": 64, "ended": 9},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    if rng.random() < 0.2:
        return {"op": "release", "batch": _log(rng, 1, 1024), "page": rng.choice((8, 16, 32, 64)), "new": _log(rng, 1, 4096),
                "lo": rng.choice((1, 77)), "hi": _log(rng, 100, 65536), "window": _log(rng, 1, 8192),
                "first": rng.choice((0, 1, 4, 100)), "ended": rng.randrange(0, 3)}
    dim = rng.choice((64, 128, 128, 256))
    hkv, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 5, 7, 8, 12))
    batch, new_hi = _log(rng, 1, 64), rng.choice((1, _log(rng, 2, 64), _log(rng, 65, 8192)))
    hi = _log(rng, 80, 32768)
    c = {"op": "stream", "fmt": rng.choice(("bf16", "bf16", "fp8", "nvfp4")), "batch": batch, "single": 0, "new_lo": 1,
         "new_hi": new_hi, "hq": hkv * group, "hkv": hkv, "dim": dim, "page": rng.choice((8, 16, 32, 64, 128)), "lo": 0,
         "hi": hi, "window": rng.choice((0, _log(rng, 1, 8192))), "first": 0}
    c["new_lo"] = _log(rng, 1, new_hi)
    if c["window"]:
        c["first"] = rng.choice((0, 1, 4, 64, 130))
    c["lo"] = rng.choice((1, _log(rng, 1, hi)))
    c["single"] = rng.randrange(0, 1 + batch)
    while c["batch"] > 1 and _too_much(c):
        c["batch"] = c["batch"] // 2
        c["single"] = min(c["single"], c["batch"])
    while _too_much(c):
        c["new_hi"] = max(1, c["new_hi"] // 2)
        c["new_lo"] = min(c["new_lo"], c["new_hi"])
        c["hi"] = max(80, c["hi"] // 2)
        c["lo"] = min(c["lo"], c["hi"])
    return c


def _too_much(c):
    """Over a fifth of a trillion operations, or over what the plain form holds at a time: scores and gathered values."""
    rows = _rows(c)
    new, most = max(n for _, n in rows), max(length for length, _ in rows)
    size = _block(new)
    blocks = sum(-(-n // size) for _, n in rows)
    keys = blocks * (min(most, (c["window"] or most) + size) + c["first"])
    return _pairs(c) * c["hq"] * c["dim"] * 4 > 2e11 or keys * c["hkv"] * c["dim"] > 1 << 30 or keys * size * c["hq"] > 1 << 32


def _spread(lo, hi, count):
    """`count` whole numbers spread evenly over the logarithm of [lo, hi]."""
    return [max(lo, min(hi, round(lo * (hi / lo) ** ((i + 0.5) / count)))) for i in range(count)]


def _rows(c):
    """(tokens with the new ones, new tokens) of every row, in a fixed order; the rows of single tokens are spread among
    the others."""
    b, single = c["batch"], c["single"]
    rest = _spread(c["new_lo"], c["new_hi"], b - single) if single < b else []
    new = sorted([((i + 0.5) / single, 1) for i in range(single)] + [((i + 0.25) / len(rest), n) for i, n in enumerate(rest)])
    return [(max(length, n), n) for length, (_, n) in zip(_spread(c["lo"], c["hi"], b), new)]


def _pairs(c):
    """(query, visible token) pairs of all rows."""
    cap, total = (c["window"] or 1 << 40) + c["first"], 0
    for length, n in _rows(c):
        full = min(n, max(0, length - cap))  # the last ones: position p sees min(p + 1, window + first) tokens
        part = n - full
        total += full * cap + part * (length - n) + part * (part + 1) // 2
    return total


def _row_bytes(fmt, dim):
    return {"bf16": 2 * dim, "fp8": dim, "nvfp4": (dim // 2 + dim // 16 + 15) // 16 * 16}[fmt]


def work(case):
    c = case
    if c["op"] == "release":
        pages = sum(_given(c, length, i) for i, length in enumerate(_lengths(c)))
        return {"bytes": 24 * c["batch"] + 12 * pages + 8, "flops": pages}
    rows = _rows(c)
    seen = [min(length, c["window"] + n - 1 + c["first"]) if c["window"] else length for length, n in rows]
    t = sum(n for _, n in rows)
    kv = 2 * sum(seen) * c["hkv"] * _row_bytes(c["fmt"], c["dim"])
    # queries, outputs, log-sum-exps, table entries
    io = t * c["hq"] * (4 * c["dim"] + 4) + 4 * sum(-(-s // c["page"]) for s in seen)
    return {"bytes": kv + io, "flops": 4 * c["hq"] * c["dim"] * _pairs(c)}


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _order(g, values):
    at = torch.randperm(len(values), generator=g, device="cuda").tolist()
    return [values[i] for i in at]


def _e2m1(x):
    """Codes (0 to 15) of the nearest 4-bit values, ties to the even code."""
    a = x.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    return code + 8 * torch.signbit(x).int()


def _to_fp8(x, scale):
    return (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _to_nvfp4(x, scale):
    """Rows of code pairs, block scales and zero padding of the values x [..., dim]."""
    dim = x.shape[-1]
    y = (x / scale).unflatten(-1, (dim // 16, 16))
    block = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    by = block.to(x.dtype)[..., None]
    code = torch.where(by > 0, _e2m1(y / torch.where(by > 0, by, 1.0)), 0).flatten(-2)
    pair = (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8)
    pad = _row_bytes("nvfp4", dim) - dim // 2 - dim // 16
    return torch.cat((pair, block.view(torch.uint8), pair.new_zeros(*pair.shape[:-1], pad)), -1)


def _values(pool, fmt, scale, dim, kind):
    """Values of gathered pool rows."""
    if fmt == "bf16":
        return pool.to(kind)
    if fmt == "fp8":
        return pool.view(torch.float8_e4m3fn).to(kind) * scale
    pair = pool[..., :dim // 2].int()
    code = torch.stack((pair & 15, pair >> 4), -1).flatten(-2).long()
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=kind, device=pool.device)[code]
    block = pool[..., dim // 2:dim // 2 + dim // 16].view(torch.float8_e4m3fn).to(kind)
    return (value.unflatten(-1, (dim // 16, 16)) * block[..., None]).flatten(-2) * scale


def _pool(g, fmt, pages, page, hkv, dim, scale):
    x = _normal(g, pages, page, hkv, dim)
    return x.to(torch.bfloat16) if fmt == "bf16" else _to_fp8(x, scale).view(torch.uint8) if fmt == "fp8" else _to_nvfp4(x, scale)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    return _prepare_release(c, g) if c["op"] == "release" else _prepare_stream(c, g)


def _prepare_stream(c, g):
    rows = _order(g, _rows(c))
    lens, n, page = [r[0] for r in rows], [r[1] for r in rows], c["page"]
    # a table over a permuted pool; pages between the first tokens and the oldest window have been given back
    kept = -(-c["first"] // page)
    gone = [max(0, (length - k + 1 - c["window"]) // page) if c["window"] else 0 for length, k in rows]
    held = [[j for j in range(-(-length // page)) if j < kept or j >= away] for length, away in zip(lens, gone)]
    total = sum(len(h) for h in held) + 3
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32).tolist()
    width = -(-max(lens) // page)
    table, at = [], 0
    for h in held:
        entries = [-1] * width
        for j in h:
            entries[j] = perm[at]
            at += 1
        table.append(entries)
    start = [0]
    for k in n:
        start.append(start[-1] + k)
    scales = {"bf16": (1.0, 1.0), "fp8": (0.02, 0.015), "nvfp4": (0.25, 0.0625)}[c["fmt"]]
    t = start[-1]
    q = _normal(g, t, c["hq"], c["dim"]).to(torch.bfloat16)
    return {"case": c, "q": q, "k": _pool(g, c["fmt"], total, page, c["hkv"], c["dim"], scales[0]),
            "v": _pool(g, c["fmt"], total, page, c["hkv"], c["dim"], scales[1]), "table": _int(table),
            "lens": _int(lens), "start": _int(start), "scales": scales, "tokens": t, "most": max(lens), "new": max(n),
            "blocks": sum(-(-k // _block(max(n))) for k in n), "out": torch.zeros_like(q),
            "lse": torch.zeros(t, c["hq"], device="cuda"), "workspace": None}


def _block(new):
    """Queries of a block of the plain form."""
    return min(new, 512)


def _lengths(c):
    return _spread(max(c["lo"], 1), max(c["hi"], c["lo"], 1), c["batch"])


def _is_ended(c, i):
    step = max(1, c["batch"] // max(1, c["ended"]))
    return i % step == 0 and i // step < c["ended"]


def _behind(c, length):
    """Pages that lie behind the windows of a row's tokens from `length` on."""
    return max(0, length + 1 - c["window"]) // c["page"]


def _given(c, length, i):
    kept, before = -(-c["first"] // c["page"]), _behind(c, length - min(length, c["new"]))
    if _is_ended(c, i):
        return -(-length // c["page"]) - max(0, before - kept)
    return max(0, _behind(c, length) - max(kept, before))


def _prepare_release(c, g):
    b, page = c["batch"], c["page"]
    kept = -(-c["first"] // page)
    rows = _order(g, list(enumerate(_lengths(c))))
    lens, ended = [length for _, length in rows], [int(_is_ended(c, i)) for i, _ in rows]
    held = _int([-(-length // page) for length in lens])
    # what the step before has given back already
    before = [_behind(c, length - min(length, c["new"])) for length in lens]
    before = _int([x if x > kept else 0 for x in before])
    width = -(-max(lens) // page) + 2
    column = torch.arange(width, device="cuda")
    there = (column < held[:, None]) & ((column < kept) | (column >= before[:, None]))
    number = (there.flatten().cumsum(0) - 1).view(b, width)
    used = int(there.sum())
    free = used // 3 + 1
    perm = torch.randperm(used + free, generator=g, device="cuda").to(torch.int32)
    table = torch.where(there, perm[number.clamp(min=0)], -1)
    free_list = torch.full((used + free,), -1, dtype=torch.int32, device="cuda")
    free_list[:free] = perm[used:]
    return {"case": c, "lens": _int(lens), "held": held, "behind": before, "ended": _int(ended), "table": table,
            "free_list": free_list, "free_count": _int([free]), "table_out": table.clone(),
            "lens_out": _int([0] * b), "held_out": _int([0] * b), "behind_out": _int([0] * b), "free_out": _int([0])}


# ---------------------------------------------------------------------------------------------- one pass

def run(state):
    if state["case"]["op"] == "release":
        return _own_release(state) if own else _release(state)
    return _own_stream(state) if own else _stream(state)


def _scale(c):
    return 1.0 / math.sqrt(c["dim"])


def _stream(s):
    """Blocks of queries of one row each: their keys are the row's first tokens and a run that ends at the last query."""
    c, dev = s["case"], s["q"].device
    hkv, d, page, most = c["hkv"], c["dim"], c["page"], s["most"]
    group, size, blocks = c["hq"] // hkv, _block(s["new"]), s["blocks"]
    window, first = (c["window"], min(c["first"], most)) if c["window"] else (1 << 30, 0)
    start, length = s["start"].long(), s["lens"].long()
    n = start[1:] - start[:-1]
    per_row = (n + size - 1) // size
    ends = per_row.cumsum(0)
    row = torch.repeat_interleave(torch.arange(n.numel(), device=dev), per_row, output_size=blocks)
    begin = (torch.arange(blocks, device=dev) - (ends - per_row)[row]) * size  # the block's first query in its row
    query = begin[:, None] + torch.arange(size, device=dev)
    real = query < n[row][:, None]
    position = (length - n)[row][:, None] + query
    index = (start[row][:, None] + query).clamp(max=s["tokens"] - 1)
    # keys: first tokens that lie before the run, then the run
    oldest = (position[:, :1] + 1 - window).clamp(min=0)
    run_length = min(most, window + size - 1)
    head = torch.arange(first, device=dev).expand(blocks, first)
    token = torch.cat((head, oldest + torch.arange(run_length, device=dev)), 1)
    twice = torch.cat((head >= oldest, torch.zeros(blocks, run_length, dtype=torch.bool, device=dev)), 1)
    seen = (token[:, None] <= position[:, :, None]) & ((token[:, None] > position[:, :, None] - window) | (token[:, None] < first))
    seen = seen & ~twice[:, None] & real[:, :, None]
    at = torch.minimum(token, length[row][:, None] - 1)
    slot = (s["table"].long()[row[:, None], at // page] * page + at % page).clamp(min=0)
    k = _values(s["k"].flatten(0, 1)[slot], c["fmt"], s["scales"][0], d, torch.float32)
    v = _values(s["v"].flatten(0, 1)[slot], c["fmt"], s["scales"][1], d, torch.float32)
    q = s["q"][index].float().view(blocks, size, hkv, group, d).permute(0, 2, 3, 1, 4)  # [blocks, hkv, group, size, d]
    score = q.reshape(blocks, hkv, group * size, d) @ k.permute(0, 2, 3, 1)
    score = score.mul_(_scale(c)).view(blocks, hkv, group, size, -1)
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(blocks, hkv, group * size, -1) @ v.transpose(1, 2)).view(blocks, hkv, group, size, d)
    out = out / torch.where(total > 0, total, 1.0)
    lse = (top + total.log())[..., 0]
    out = out.permute(0, 3, 1, 2, 4).reshape(blocks, size, c["hq"], d)[real]
    lse = lse.permute(0, 3, 1, 2).reshape(blocks, size, c["hq"])[real]
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _release(s):
    c, dev = s["case"], s["lens"].device
    page, kept, width = c["page"], -(-c["first"] // c["page"]), s["table"].shape[1]
    lens, held, before, ended = s["lens"].long(), s["held"].long(), s["behind"].long(), s["ended"] > 0
    behind = torch.minimum((lens + 1 - c["window"]).clamp(min=0) // page, held)
    after = torch.maximum(before, torch.where(behind > kept, behind, 0))
    column = torch.arange(width, device=dev)
    gone = (column >= kept) & (column < before[:, None])
    give = torch.where(ended[:, None], column < held[:, None], (column >= kept) & (column < after[:, None])) & ~gone
    count = s["free_count"].long()
    to = count + give.flatten().cumsum(0) - 1
    spare = s["free_list"].numel()
    padded = torch.cat((s["free_list"], s["free_list"].new_zeros(1)))
    padded[torch.where(give.flatten(), to, spare)] = torch.where(give, s["table"], 0).flatten()
    s["free_list"].copy_(padded[:spare])
    s["table_out"].copy_(torch.where(give, -1, s["table"]))
    s["lens_out"].copy_(torch.where(ended, 0, lens))
    s["held_out"].copy_(torch.where(ended, 0, held))
    s["behind_out"].copy_(torch.where(ended, 0, after))
    s["free_out"].copy_(count + give.sum())
    return _released(s)


def _released(s):
    return [s[k] for k in ("free_list", "free_out", "table_out", "lens_out", "held_out", "behind_out")]


# ---------------------------------------------------------------------------------------------- the framework's calls

def _own_stream(s):
    import paged_kv_attention_19_gb300 as pa
    c = s["case"]
    if s["workspace"] is None:
        s["workspace"] = pa.workspace_for_stream(s["q"], s["k"], s["table"], s["new"])
    more = {} if c["fmt"] == "bf16" else {"k_scale": s["scales"][0], "v_scale": s["scales"][1]}
    call = {"bf16": pa.pa_stream_gqa, "fp8": pa.pa_stream_gqa_fp8, "nvfp4": pa.pa_stream_gqa_nvfp4}[c["fmt"]]
    call(s["q"], s["k"], s["v"], s["table"], s["lens"], s["start"], s["out"], s["lse"], max_query=s["new"],
         scale=_scale(c), window=c["window"], first=c["first"], workspace=s["workspace"], **more)
    return {"out": s["out"], "lse": s["lse"]}


def _own_release(s):
    import paged_kv_attention_19_gb300 as pa
    c = s["case"]
    pa.pa_release_pages(s["lens"], s["held"], s["behind"], s["free_list"], s["free_count"], s["table"], page_size=c["page"],
                        window=c["window"], first=c["first"], ended=s["ended"], context_lens_out=s["lens_out"],
                        held_pages_out=s["held_out"], window_start_out=s["behind_out"], free_count_out=s["free_out"],
                        block_table_out=s["table_out"])
    return _released(s)


# ---------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """Row by row from the definition: the token at position p sees those of [0, p] that are among the row's `first`
    tokens or less than `window` back."""
    if case["op"] == "release":
        return None  # whole numbers: nothing is computed
    s = prepare(case, seed)
    c, d, page, group = s["case"], case["dim"], case["page"], case["hq"] // case["hkv"]
    out = torch.zeros(s["tokens"], c["hkv"], group, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["tokens"], c["hkv"], group, dtype=torch.float64, device="cuda")
    start, lens = s["start"].tolist(), s["lens"].tolist()
    for b, length in enumerate(lens):
        for q0 in range(start[b], start[b + 1], 1024):
            q1 = min(q0 + 1024, start[b + 1])
            p = torch.arange(q0, q1, device="cuda") + (length - start[b + 1])
            p0, p1 = length - start[b + 1] + q0, length - start[b + 1] + q1 - 1
            low = max(0, p0 - c["window"] + 1) if c["window"] else 0
            tokens = torch.cat((torch.arange(min(c["first"], low), device="cuda"), torch.arange(low, p1 + 1, device="cuda")))
            allowed = tokens <= p[:, None]
            if c["window"]:
                allowed &= (p[:, None] - tokens < c["window"]) | (tokens < c["first"])
            rows = s["table"][b, tokens // page].long(), tokens % page
            k = _values(s["k"][rows], c["fmt"], s["scales"][0], d, torch.float64)
            v = _values(s["v"][rows], c["fmt"], s["scales"][1], d, torch.float64)
            q = s["q"][q0:q1].double().view(q1 - q0, c["hkv"], group, d)
            for h in range(c["hkv"]):
                score = torch.einsum("ngd,ld->ngl", q[:, h], k[:, h]) / math.sqrt(d)
                score = score.masked_fill(~allowed[:, None], -math.inf)
                out[q0:q1, h] = torch.softmax(score, -1) @ v[:, h]
                lse[q0:q1, h] = torch.logsumexp(score, -1)
    return {"out": out.flatten(1, 2), "lse": lse.flatten(1, 2)}
