"""Timed cases of the operators around tree-drafted decoding over the paged cache.

One decoding step with drafted trees is four operators, and each case below is one call of one of them:
  plan      pages, block tables, slots, positions and tree masks of a step's new tokens
  rope      norms of queries and keys for each head, position rotation, and the write into the paged cache
  tree      attention of every row's drafted tree over its paged context and its own ancestors
  compact   moves the accepted path's keys and values together, so that they are the row's newest tokens

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
        # one request, a short tree: the latency of a single user's step
        {"name": "tree-bf16-single", "op": "tree", "fmt": "bf16", "batch": 1, "nodes": 8, "ragged": False, "hq": 32,
         "hkv": 8, "dim": 128, "page": 16, "lo": 1000, "hi": 1000, "window": 0},
        # the widest trees (64 nodes, 512 query rows for each key head) at a moderate batch
        {"name": "tree-bf16-wide", "op": "tree", "fmt": "bf16", "batch": 16, "nodes": 64, "ragged": False, "hq": 64,
         "hkv": 8, "dim": 128, "page": 32, "lo": 1024, "hi": 8192, "window": 0},
        # ragged trees in a sliding-window layer with wide heads
        {"name": "tree-bf16-window", "op": "tree", "fmt": "bf16", "batch": 16, "nodes": 13, "ragged": True, "hq": 16,
         "hkv": 4, "dim": 256, "page": 32, "lo": 2048, "hi": 32768, "window": 4096},
        # serving at concurrency over an 8-bit cache, ragged trees, long and short contexts together
        {"name": "tree-fp8-serving", "op": "tree", "fmt": "fp8", "batch": 32, "nodes": 16, "ragged": True, "hq": 64,
         "hkv": 8, "dim": 128, "page": 32, "lo": 128, "hi": 16384, "window": 0},
        # the same over a 4-bit cache
        {"name": "tree-nvfp4-serving", "op": "tree", "fmt": "nvfp4", "batch": 32, "nodes": 16, "ragged": True,
         "hq": 64, "hkv": 8, "dim": 128, "page": 32, "lo": 128, "hi": 16384, "window": 0},
        # a small batch's decode step
        {"name": "rope-bf16-decode", "op": "rope", "fmt": "bf16", "tokens": 61, "pad": 3, "hq": 32, "hkv": 8,
         "dim": 128, "rot": 128, "interleaved": False, "page": 16, "far": 40000},
        # a prefill chunk into an 8-bit cache
        {"name": "rope-fp8-prefill", "op": "rope", "fmt": "fp8", "tokens": 8192, "pad": 0, "hq": 64, "hkv": 8,
         "dim": 128, "rot": 128, "interleaved": False, "page": 32, "far": 131072},
        # a chunk into a 4-bit cache, half of wide heads rotated, adjacent pairs
        {"name": "rope-nvfp4-partial", "op": "rope", "fmt": "nvfp4", "tokens": 2011, "pad": 37, "hq": 16, "hkv": 4,
         "dim": 256, "rot": 128, "interleaved": True, "page": 32, "far": 32768},
        # a decode step's plan: every row drafts a tree, some rows have ended
        {"name": "plan-trees", "op": "plan", "batch": 48, "page": 32, "lo": 128, "hi": 16384, "new_lo": 1,
         "new_hi": 64, "ended": 5, "tree": True, "scarce": False},
        # decodes mixed with prefill chunks, the free list too short for all of them
        {"name": "plan-mixed-scarce", "op": "plan", "batch": 512, "page": 16, "lo": 1, "hi": 32768, "new_lo": 1,
         "new_hi": 1024, "ended": 31, "tree": False, "scarce": True},
        # one layer's accepted rows
        {"name": "compact-layer", "op": "compact", "fmt": "bf16", "layers": 1, "batch": 32, "nodes": 16,
         "accepted": 5, "hkv": 8, "dim": 128, "page": 32, "lo": 128, "hi": 4096},
        # every layer of an 8-bit cache in one call
        {"name": "compact-layers-fp8", "op": "compact", "fmt": "fp8", "layers": 48, "batch": 64, "nodes": 63,
         "accepted": 9, "hkv": 8, "dim": 128, "page": 16, "lo": 64, "hi": 512},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "tree", "rope", "rope", "plan", "compact"))
    if op == "tree":
        dim = rng.choice((64, 128, 128, 256))
        fmt = rng.choice(("bf16", "bf16", "fp8", "nvfp4") if dim > 64 else ("bf16", "nvfp4"))
        hkv = rng.choice((1, 2, 4, 8))
        group = rng.choice((1, 2, 3, 4, 5, 7, 8, 12))
        batch, nodes = _log(rng, 1, 32), _log(rng, 1, 64)
        while batch * nodes * group > 4096:
            batch = max(1, batch // 2)
        hi = _log(rng, 80, min(16384, max(80, 262144 // batch)))
        return {"op": op, "fmt": fmt, "batch": batch, "nodes": nodes, "ragged": rng.random() < 0.5,
                "hq": hkv * group, "hkv": hkv, "dim": dim, "page": rng.choice((8, 16, 32, 64, 128)),
                "lo": _log(rng, nodes, hi) if hi > nodes else nodes, "hi": max(hi, nodes),
                "window": rng.choice((0, 0, _log(rng, 1, 8192)))}
    if op == "rope":
        dim = rng.choice((64, 128, 128, 256))
        hkv = rng.choice((1, 2, 4, 8))
        tokens = _log(rng, 1, 4096)
        return {"op": op, "fmt": rng.choice(("bf16", "fp8", "nvfp4")), "tokens": tokens,
                "pad": rng.randrange(0, 1 + tokens // 8), "hq": hkv * rng.choice((1, 2, 4, 5, 8)), "hkv": hkv,
                "dim": dim, "rot": rng.choice((dim, dim, dim // 2)), "interleaved": rng.random() < 0.4,
                "page": rng.choice((8, 16, 32, 64)), "far": _log(rng, 64, 131072)}
    if op == "plan":
        tree = rng.random() < 0.5
        batch, hi = _log(rng, 1, 512), _log(rng, 16, 32768)
        return {"op": op, "batch": batch, "page": rng.choice((8, 16, 32, 64, 256)), "lo": rng.choice((1, 7)),
                "hi": hi, "new_lo": 1, "new_hi": _log(rng, 1, 64 if tree else 1024), "ended": rng.randrange(0, 1 + batch // 4),
                "tree": tree, "scarce": rng.random() < 0.4}
    nodes = _log(rng, 3, 64)
    layers = _log(rng, 1, 32)
    return {"op": op, "fmt": rng.choice(("bf16", "fp8")), "layers": layers, "batch": _log(rng, 1, 64), "nodes": nodes,
            "accepted": rng.randrange(2, max(3, nodes // 2)), "hkv": rng.choice((1, 2, 4, 8)),
            "dim": rng.choice((64, 128, 256)), "page": rng.choice((8, 16, 32, 64)), "lo": 64, "hi": _log(rng, 64, 512)}


def _spread(lo, hi, count):
    """`count` whole numbers spread evenly over the logarithm of [lo, hi]."""
    return [max(lo, min(hi, round(lo * (hi / lo) ** ((i + 0.5) / count)))) for i in range(count)]


def _rows(c):
    """(context length with the new tokens, nodes) of every row of a tree or compact case, in a fixed order."""
    b, q = c["batch"], c["nodes"]
    if c["op"] == "compact":
        n = [q] * b
    else:
        n = [1 + (i * 5 + 2) % q if c["ragged"] else q for i in range(b)]
    return [(max(length, k), k) for length, k in zip(_spread(c["lo"], c["hi"], b), n)]


def _news(c):
    """New tokens of every row of a plan case (-1: the row has ended), in a fixed order."""
    n = _spread(c["new_lo"], c["new_hi"], c["batch"])
    step = max(1, c["batch"] // max(1, c["ended"]))
    left = c["ended"]
    for i in range(0, c["batch"], step):
        if left > 0:
            n[i], left = -1, left - 1
    return n


def _row_bytes(fmt, dim):
    return {"bf16": 2 * dim, "fp8": dim, "nvfp4": (dim // 2 + dim // 16 + 15) // 16 * 16}[fmt]


def work(case):
    c = case
    if c["op"] == "tree":
        rows = _rows(c)
        seen = [min(length, c["window"] + k) if c["window"] else length for length, k in rows]
        t = sum(k for _, k in rows)
        kv = 2 * sum(seen) * c["hkv"] * _row_bytes(c["fmt"], c["dim"])
        # queries, outputs, log-sum-exps, masks, table entries
        io = t * c["hq"] * (4 * c["dim"] + 4) + 8 * t + 4 * sum(-(-s // c["page"]) for s in seen)
        return {"bytes": kv + io, "flops": 4 * c["hq"] * c["dim"] * sum(s * k for s, (_, k) in zip(seen, rows))}
    if c["op"] == "rope":
        t, d = c["tokens"], c["dim"]
        read = t * (c["hq"] + 2 * c["hkv"]) * 2 * d + t * (12 + 4 * c["rot"])
        written = t * c["hq"] * 2 * d + 2 * t * c["hkv"] * _row_bytes(c["fmt"], d)
        return {"bytes": read + written, "flops": t * (c["hq"] + c["hkv"]) * 8 * d}
    if c["op"] == "plan":
        news = _news(c)
        t = sum(max(0, n) for n in news)
        pages = sum(max(0, n) // c["page"] for n in news)
        return {"bytes": c["batch"] * 24 + t * (12 + (12 if c["tree"] else 0)) + 8 * pages + 8 * c["batch"], "flops": t}
    moved = sum(m - 1 for m in _accepted(c))
    return {"bytes": 4 * moved * c["layers"] * c["hkv"] * _row_bytes(c["fmt"], c["dim"]) + 16 * c["batch"], "flops": 0}


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tables(g, lens, page, most):
    """A block table for rows of up to `most` tokens over a permuted pool, and the pool's pages."""
    pages = [-(-n // page) for n in lens]
    total = sum(pages) + 3
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), -(-most // page), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total


def _parents(g, rows, nodes):
    """Random recursive trees: node 0 is the root, node i hangs below an earlier one."""
    at = torch.arange(nodes, device="cuda")
    u = torch.rand(rows, nodes, generator=g, device="cuda")
    return torch.where(at > 0, torch.minimum((u * at).long(), (at - 1).clamp(min=0)), -1).to(torch.int32)


def _wider(reach):
    return ((reach @ reach) > 0).float()


def _ancestors(parents):
    """[rows, nodes, nodes] truth: node j is node i or one of its ancestors."""
    rows, nodes = parents.shape
    at = torch.arange(nodes, device=parents.device)
    reach = (parents[:, :, None] == at) | (at[:, None] == at)
    return _wider(_wider(_wider(_wider(_wider(_wider(reach.float())))))) > 0


def _bits(reach):
    at = torch.arange(reach.shape[-1], device=reach.device)
    return torch.where(reach, torch.ones((), dtype=torch.int64, device=reach.device) << at, 0).sum(-1)


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


def _from_pool(pool, fmt, scale, dim, kind):
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


def _accepted(c):
    return [1 + i % c["accepted"] if c["batch"] > 1 else c["accepted"] for i in range(c["batch"])]


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    return {"tree": _prepare_tree, "rope": _prepare_rope, "plan": _prepare_plan, "compact": _prepare_compact}[c["op"]](c, g)


def _order(g, values):
    at = torch.randperm(len(values), generator=g, device="cuda").tolist()
    return [values[i] for i in at]


def _prepare_tree(c, g):
    rows = _order(g, _rows(c))
    lens, n = [r[0] for r in rows], [r[1] for r in rows]
    table, pages = _tables(g, lens, c["page"], max(lens))
    start = [0]
    for k in n:
        start.append(start[-1] + k)
    reach = _ancestors(_parents(g, c["batch"], c["nodes"]))
    at = torch.cat([torch.arange(k, device="cuda") + b * c["nodes"] for b, k in enumerate(n)])
    # a node's mask never names nodes behind the row's own: they come after it in the tree's order
    mask = _bits(reach).reshape(-1)[at].contiguous()
    scales = {"bf16": (1.0, 1.0), "fp8": (0.02, 0.015), "nvfp4": (0.25, 0.0625)}[c["fmt"]]
    t = start[-1]
    q = _normal(g, t, c["hq"], c["dim"]).to(torch.bfloat16)
    return {"case": c, "q": q, "k": _pool(g, c["fmt"], pages, c["page"], c["hkv"], c["dim"], scales[0]),
            "v": _pool(g, c["fmt"], pages, c["page"], c["hkv"], c["dim"], scales[1]), "table": table,
            "lens": _int(lens), "start": _int(start), "mask": mask, "scales": scales, "tokens": t, "most": max(lens),
            "out": torch.zeros_like(q), "lse": torch.zeros(t, c["hq"], device="cuda"), "workspace": None}


def _prepare_rope(c, g):
    t, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["dim"]
    pages = -(-t * 5 // (4 * c["page"])) + 1
    # queries, keys and values side by side, as one projection leaves them
    qkv = (_normal(g, t, hq + 2 * hkv, d) * 2.0).to(torch.bfloat16)
    slots = torch.randperm(pages * c["page"], generator=g, device="cuda")[:t]
    slots[t - c["pad"]:] = -1
    positions = torch.randint(0, c["far"], (t,), generator=g, device="cuda").to(torch.int32)
    angle = torch.arange(c["far"], device="cuda", dtype=torch.float64)[:, None] * (
        1e6 ** (-torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64) * 2.0 / c["rot"]))
    cos_sin = torch.cat((angle.cos(), angle.sin()), -1).float()
    weights = [(1.0 + 0.1 * _normal(g, d)).to(torch.bfloat16) for _ in range(2)]
    scales = {"bf16": (1.0, 1.0), "fp8": (0.011, 0.021), "nvfp4": (0.25, 0.0625)}[c["fmt"]]
    kind = torch.bfloat16 if c["fmt"] == "bf16" else torch.uint8
    width = d if c["fmt"] != "nvfp4" else _row_bytes("nvfp4", d)
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    byte = torch.arange(256, device="cuda")
    both = torch.stack((lut[byte & 15], lut[byte >> 4]), -1).contiguous().view(torch.int16).flatten()
    k_pool = torch.zeros(pages, c["page"], hkv, width, dtype=kind, device="cuda")
    return {"case": c, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:], "wq": weights[0],
            "wk": weights[1], "cos_sin": cos_sin, "positions": positions, "slots": slots, "scales": scales,
            "q_out": torch.zeros(t, hq, d, dtype=torch.bfloat16, device="cuda"), "k_pool": k_pool,
            "v_pool": torch.zeros_like(k_pool), "values": both}


def _prepare_plan(c, g):
    b, p = c["batch"], c["page"]
    news, lens = _news(c), _spread(c["lo"], c["hi"], c["batch"])
    lens = _order(g, lens)
    held = [-(-n // p) for n in lens]
    at = torch.randint(0, 3, (b,), generator=g, device="cuda").tolist()
    held = [h + (1 if a == 0 else 0) for h, a in zip(held, at)]  # pages left over from rejected drafts
    need = [max(0, -(-(n + k) // p) - h) if k >= 0 else 0 for n, k, h in zip(lens, news, held)]
    free = sum(need) // (2 if c["scarce"] else 1) + (0 if c["scarce"] else 7)
    total = sum(-(-n // p) + 2 for n in lens) + sum(-(-max(0, k) // p) for k in news) + 7
    width = -(-(c["hi"] + c["new_hi"]) // p) + 2
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    used = 0
    for i, h in enumerate(held):
        table[i, :h] = perm[used:used + h]
        used += h
    free_list = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    free_list[:free] = perm[used:used + free]
    t = sum(max(0, k) for k in news)
    tokens = t + 13  # a padded batch
    parents = None
    if c["tree"]:
        grid = _parents(g, b, 64)
        parents = torch.cat([grid[i, :k] for i, k in enumerate(news) if k > 0] + [_int([-1] * 13)]).contiguous()
    return {"case": c, "lens": _int(lens), "news": _int(news), "held": _int(held), "free_list": free_list,
            "free_count": _int([free]), "table": table, "parents": parents, "pages": total,
            "lens_out": torch.zeros(b, dtype=torch.int32, device="cuda"),
            "held_out": torch.zeros(b, dtype=torch.int32, device="cuda"), "free_out": _int([0]),
            "start": torch.zeros(b + 1, dtype=torch.int32, device="cuda"),
            "slots": torch.zeros(tokens, dtype=torch.int64, device="cuda"),
            "positions": torch.zeros(tokens, dtype=torch.int32, device="cuda"),
            "mask": torch.zeros(tokens, dtype=torch.int64, device="cuda") if c["tree"] else None}


def _prepare_compact(c, g):
    rows = _rows(c)
    lens, b, m = _order(g, [r[0] for r in rows]), c["batch"], c["accepted"]
    table, pages = _tables(g, lens, c["page"], max(lens))
    counts = _int(_order(g, _accepted(c)))
    extra = torch.randint(1, c["nodes"] - m + 1, (b, m - 1), generator=g, device="cuda").sort(-1).values
    path = torch.cat((extra.new_zeros(b, 1), extra + torch.arange(1, m, device="cuda")), -1).to(torch.int32)
    path = torch.where(torch.arange(m, device="cuda") < counts[:, None], path, -1)
    shape = (c["layers"], pages, c["page"], c["hkv"], c["dim"])
    if c["fmt"] == "bf16":
        k, v = (torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    else:
        k, v = (torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
    start = torch.arange(b + 1, dtype=torch.int32, device="cuda") * c["nodes"]
    return {"case": c, "k": k, "v": v, "table": table, "lens": _int(lens), "start": start, "path": path,
            "counts": counts, "lens_out": torch.zeros(b, dtype=torch.int32, device="cuda")}


# ---------------------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree": _own_tree, "rope": _own_rope, "plan": _own_plan, "compact": _own_compact}[op](state)
    return {"tree": _tree, "rope": _rope, "plan": _plan, "compact": _compact}[op](state)


def _scale(c):
    return 1.0 / math.sqrt(c["dim"])


def _tree(s):
    c = s["case"]
    b, n_max, hkv, d, page, most = c["batch"], c["nodes"], c["hkv"], c["dim"], c["page"], s["most"]
    group = c["hq"] // hkv
    start, dev = s["start"].long(), s["q"].device
    n = start[1:] - start[:-1]
    node = torch.arange(n_max, device=dev)
    index = (start[:-1, None] + node).clamp(max=s["tokens"] - 1)
    real = node < n[:, None]
    q = s["q"][index].float().view(b, n_max, hkv, group, d).transpose(1, 2).reshape(b, hkv, n_max * group, d)
    token = torch.arange(most, device=dev)
    slot = s["table"].long()[:, token // page] * page + token % page
    k = _from_pool(s["k"].flatten(0, 1)[slot], c["fmt"], s["scales"][0], d, torch.float32)
    v = _from_pool(s["v"].flatten(0, 1)[slot], c["fmt"], s["scales"][1], d, torch.float32)
    mask = torch.where(real, s["mask"][index], 0)
    reach = ((mask[:, :, None] >> node) & 1) > 0
    depth = (reach & (node[:, None] != node)).sum(-1)
    length = s["lens"].long()[:, None, None]
    prefix = length - n[:, None, None]
    window = c["window"] if c["window"] else 1 << 30
    reach = reach & (depth[:, :, None] - depth[:, None, :] < window)
    drafted = reach.gather(2, (token - prefix).clamp(0, n_max - 1).expand(b, n_max, most))
    seen = torch.where(token < prefix, prefix + depth[:, :, None] - token < window, drafted & (token < length))
    seen = seen[:, None, :, None].expand(b, 1, n_max, group, most).reshape(b, 1, n_max * group, most)
    score = (q @ k.permute(0, 2, 3, 1)) * _scale(c)
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    out = (p @ v.transpose(1, 2)) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log())[..., 0]
    t = torch.arange(s["tokens"], device=dev)
    row = (t[:, None] >= start[1:]).sum(1)
    at = t - start[row]
    out = out.view(b, hkv, n_max, group, d).transpose(1, 2).reshape(b, n_max, c["hq"], d)[row, at]
    lse = lse.view(b, hkv, n_max, group).transpose(1, 2).reshape(b, n_max, c["hq"])[row, at]
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _rotated(x, weight, cos, sin, rot, interleaved):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _stored(x, fmt, scale):
    return x.to(torch.bfloat16) if fmt == "bf16" else _to_fp8(x, scale).view(torch.uint8) if fmt == "fp8" else _to_nvfp4(x, scale)


def _held(s, pool):
    """A pool as the values that it holds."""
    c = s["case"]
    if c["fmt"] == "bf16":
        return pool
    if c["fmt"] == "fp8":
        return pool.view(torch.float8_e4m3fn)
    d = c["dim"]
    value = s["values"][pool[..., :d // 2].int()].view(torch.float8_e4m3fn)
    return {"values": value, "blocks": pool[..., d // 2:d // 2 + d // 16].view(torch.float8_e4m3fn)}


def _rope(s):
    c = s["case"]
    t, rot = c["tokens"] - c["pad"], c["rot"]
    angle = s["cos_sin"][s["positions"][:t].long()]
    cos, sin = angle[:, None, :rot // 2], angle[:, None, rot // 2:]
    s["q_out"][:t] = _rotated(s["q"][:t], s["wq"], cos, sin, rot, c["interleaved"]).to(torch.bfloat16)
    k = _rotated(s["k"][:t], s["wk"], cos, sin, rot, c["interleaved"])
    s["k_pool"].flatten(0, 1)[s["slots"][:t]] = _stored(k, c["fmt"], s["scales"][0])
    s["v_pool"].flatten(0, 1)[s["slots"][:t]] = _stored(s["v"][:t].float(), c["fmt"], s["scales"][1])
    return {"q": s["q_out"], "k": _held(s, s["k_pool"]), "v": _held(s, s["v_pool"])}


def _plan(s):
    c = s["case"]
    p, dev = c["page"], s["lens"].device
    lens, news, held, width = s["lens"].long(), s["news"].long(), s["held"].long(), s["table"].shape[1]
    ended, n, count = news < 0, news.clamp(min=0), s["free_count"].long()
    start = torch.cat((n.new_zeros(1), n.cumsum(0)))
    # ended rows' pages go on top of the free list
    given = torch.where(ended, held, 0)
    given_at = given.cumsum(0) - given
    column = torch.arange(width, device=dev)
    free_list = torch.cat((s["free_list"], s["free_list"].new_zeros(1)))
    spare = s["free_list"].numel()
    to = torch.where(column < given[:, None], count + given_at[:, None] + column, spare)
    free_list[to] = torch.where(to < spare, s["table"], 0)
    top = count + given.sum()
    # pages are taken from the top in row order, while they last
    need = torch.where(ended, 0, ((lens + n + p - 1) // p - held).clamp(min=0))
    through = need.cumsum(0)
    granted = ~ended & ((need == 0) | (through <= top))
    taken = torch.where(granted, need, 0)
    into = (column >= held[:, None]) & (column < (held + taken)[:, None])
    source = (top - 1 - (through - need)[:, None] - (column - held[:, None])).clamp(0, spare)
    s["table"].copy_(torch.where(into, free_list[source], s["table"]))
    s["free_list"].copy_(free_list[:spare])
    s["lens_out"].copy_(torch.where(ended, 0, torch.where(granted, lens + n, lens)))
    s["held_out"].copy_(torch.where(ended, 0, held + taken))
    s["free_out"].copy_(top - taken.sum())
    s["start"].copy_(start)
    # the new tokens
    t = torch.arange(s["slots"].numel(), device=dev)
    row = (t[:, None] >= start[1:]).sum(1)
    inside = row < c["batch"]
    row = row.clamp(max=c["batch"] - 1)
    i = t - start[row]
    at = lens[row] + i
    page = s["table"][row, (at // p).clamp(max=width - 1)].long()
    s["slots"].copy_(torch.where(inside & granted[row], page * p + at % p, -1))
    if c["tree"]:
        node = torch.arange(64, device=dev)
        pick = (start[:-1, None] + node).clamp(max=t.numel() - 1)
        parents = torch.where(node < n[:, None], s["parents"][pick], -1)
        bits = _bits(_ancestors(parents))
        depth = _ancestors(parents).sum(-1) - 1
        k = i.clamp(0, 63)
        s["mask"].copy_(torch.where(inside, bits[row, k], 0))
        at = lens[row] + depth[row, k]
    s["positions"].copy_(torch.where(inside, at, 0))
    return _planned(s)


def _planned(s):
    return [s[k] for k in ("table", "free_list", "lens_out", "held_out", "free_out", "start", "slots", "positions", "mask")]


def _compact(s):
    c, p = s["case"], s["case"]["page"]
    n = (s["start"][1:] - s["start"][:-1]).long()
    prefix = s["lens"].long() - n
    at = torch.arange(c["accepted"], device=n.device)
    moved = at < s["counts"][:, None]
    # the places behind a row's accepted path copy its first node onto itself
    source = prefix[:, None] + torch.where(moved, s["path"].long(), 0)
    target = prefix[:, None] + torch.where(moved, at, 0)
    table = s["table"].long()
    source = table.gather(1, source // p) * p + source % p
    target = table.gather(1, target // p) * p + target % p
    k, v = s["k"].flatten(1, 2), s["v"].flatten(1, 2)
    k[:, target] = k[:, source]
    v[:, target] = v[:, source]
    s["lens_out"].copy_(prefix + s["counts"])
    return _compacted(s)


def _compacted(s):
    whole = torch.int16 if s["case"]["fmt"] == "bf16" else torch.uint8
    return [s["k"].view(whole), s["v"].view(whole), s["lens_out"]]


# ---------------------------------------------------------------------------------------------- the framework's calls

def _own_tree(s):
    import paged_kv_attention_19_gb300 as pa
    c = s["case"]
    if s["workspace"] is None:
        s["workspace"] = pa.workspace_for_tree(s["q"], s["k"], s["table"], c["nodes"])
    more = {} if c["fmt"] == "bf16" else {"k_scale": s["scales"][0], "v_scale": s["scales"][1]}
    call = {"bf16": pa.pa_tree_gqa, "fp8": pa.pa_tree_gqa_fp8, "nvfp4": pa.pa_tree_gqa_nvfp4}[c["fmt"]]
    call(s["q"], s["k"], s["v"], s["table"], s["lens"], s["start"], s["mask"], s["out"], s["lse"], max_query=c["nodes"],
         scale=_scale(c), window=c["window"], workspace=s["workspace"], **more)
    return {"out": s["out"], "lse": s["lse"]}


def _own_rope(s):
    import paged_kv_attention_19_gb300 as pa
    c = s["case"]
    more = {} if c["fmt"] == "bf16" else {"k_scale": s["scales"][0], "v_scale": s["scales"][1]}
    call = {"bf16": pa.pa_qk_norm_rope_write, "fp8": pa.pa_qk_norm_rope_write_fp8,
            "nvfp4": pa.pa_qk_norm_rope_write_nvfp4}[c["fmt"]]
    call(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos_sin"], s["positions"], s["slots"], s["q_out"], s["k_pool"],
         s["v_pool"], eps=1e-6, interleaved=c["interleaved"], **more)
    return {"q": s["q_out"], "k": _held(s, s["k_pool"]), "v": _held(s, s["v_pool"])}


def _own_plan(s):
    import paged_kv_attention_19_gb300 as pa
    pa.pa_plan_step(s["lens"], s["news"], s["held"], s["free_list"], s["free_count"], s["table"], s["start"], s["slots"],
                    s["positions"], page_size=s["case"]["page"], context_lens_out=s["lens_out"],
                    held_pages_out=s["held_out"], free_count_out=s["free_out"], parents=s["parents"],
                    tree_mask=s["mask"])
    return _planned(s)


def _own_compact(s):
    import paged_kv_attention_19_gb300 as pa
    pa.pa_kv_compact(s["k"], s["v"], s["table"], s["lens"], s["start"], s["path"], s["counts"],
                     context_lens_out=s["lens_out"])
    return _compacted(s)


# ---------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(s)
    if case["op"] == "rope":
        return _exact_rope(s)
    return None  # whole numbers and copied bits: nothing is computed


def _exact_tree(s):
    """Row by row from the definition: each node attends to the row's tokens before the tree and to the nodes that its
    mask names, those fewer than `window` positions back."""
    c = s["case"]
    d, page, group = c["dim"], c["page"], c["hq"] // c["hkv"]
    out = torch.zeros(s["tokens"], c["hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["tokens"], c["hq"], dtype=torch.float64, device="cuda")
    start, lens, masks = s["start"].tolist(), s["lens"].tolist(), s["mask"].tolist()
    for b in range(c["batch"]):
        n, length = start[b + 1] - start[b], lens[b]
        prefix = length - n
        at = torch.arange(length, device="cuda")
        rows = s["table"][b, at // page].long(), at % page
        k = _from_pool(s["k"][rows], c["fmt"], s["scales"][0], d, torch.float64).repeat_interleave(group, 1)
        v = _from_pool(s["v"][rows], c["fmt"], s["scales"][1], d, torch.float64).repeat_interleave(group, 1)
        own_masks = [m & ((1 << 64) - 1) for m in masks[start[b]:start[b + 1]]]
        depth = [bin(m & ~(1 << i)).count("1") for i, m in enumerate(own_masks)]
        allowed = torch.zeros(n, length, dtype=torch.bool)
        for i, m in enumerate(own_masks):
            first = max(0, prefix + depth[i] - c["window"] + 1) if c["window"] else 0
            allowed[i, first:prefix] = True
            for j in range(n):
                if m >> j & 1 and (not c["window"] or depth[i] - depth[j] < c["window"]):
                    allowed[i, prefix + j] = True
        q = s["q"][start[b]:start[b + 1]].double()
        score = torch.einsum("nhd,lhd->hnl", q, k) * _scale(c)
        score = score.masked_fill(~allowed.cuda(), -math.inf)
        out[start[b]:start[b + 1]] = torch.einsum("hnl,lhd->nhd", torch.softmax(score, -1), v)
        lse[start[b]:start[b + 1]] = torch.logsumexp(score, -1).T
    return {"out": out, "lse": lse}


def _exact_rope(s):
    c = s["case"]
    t, d, rot = c["tokens"] - c["pad"], c["dim"], c["rot"]
    table = s["cos_sin"].double()[s["positions"][:t].long()]
    turn = torch.complex(table[:, :rot // 2], table[:, rot // 2:])[:, None]

    def turned(x, w):
        x = x[:t].double()
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + 1e-6) * w.double()
        i = torch.arange(rot // 2, device="cuda")
        first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def held(pool, x, scale):
        rows = torch.zeros(pool.shape[0] * pool.shape[1], c["hkv"], d, dtype=torch.float64, device="cuda")
        shape = (*pool.shape[:3], d)
        if c["fmt"] == "bf16":
            rows[s["slots"][:t]] = x
            return rows.view(shape)
        y = x / scale
        if c["fmt"] == "fp8":
            rows[s["slots"][:t]] = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).double()
            return rows.view(shape)
        y = y.unflatten(-1, (d // 16, 16))
        block = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).double()
        steps = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        ratio = torch.where(block[..., None] > 0, y / block[..., None].clamp(min=2.0 ** -9), 0.0)
        # the nearest step, the even one of two equally near
        apart = (ratio.abs()[..., None] - steps).abs() + (torch.arange(8, device="cuda") % 2) * 1e-13
        value = steps[apart.argmin(-1)] * torch.sign(ratio)
        rows[s["slots"][:t]] = value.flatten(-2)
        blocks = torch.zeros(rows.shape[0], c["hkv"], d // 16, dtype=torch.float64, device="cuda")
        blocks[s["slots"][:t]] = block
        return {"values": rows.view(shape), "blocks": blocks.view(*shape[:3], d // 16)}

    q = torch.zeros(c["tokens"], c["hq"], d, dtype=torch.float64, device="cuda")
    q[:t] = turned(s["q"], s["wq"])
    return {"q": q, "k": held(s["k_pool"], turned(s["k"], s["wk"]), s["scales"][0]),
            "v": held(s["v_pool"], s["v"][:t].double(), s["scales"][1])}
