"""Plain references (numpy, 64 bits) of the tree-drafting operators, and the inputs of their tests.
Test infrastructure; shares no code with the library."""
from __future__ import annotations

import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_table():
    """Values of the 256 E4M3 codes (0x7F and 0xFF: NaN)."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = math.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


def row_bytes(fmt, D):
    return {"bf16": 2 * D, "fp8": D, "nvfp4": (D // 2 + D // 16 + 15) // 16 * 16}[fmt]


def bf16_values(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def pool_values(pool, fmt, D, scale):
    """Values of a pool given as its raw array (uint16 bf16 bits, or uint8)."""
    if fmt == "bf16":
        return bf16_values(pool)
    if fmt == "fp8":
        return e4m3_table()[pool] * scale
    c = pool[..., :D // 2]
    code = np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], D)
    val = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    blk = e4m3_table()[pool[..., D // 2:D // 2 + D // 16]]
    return val * np.repeat(blk, 16, -1) * scale


def random_tree(rng, n, chain=False):
    """Parents (-1: root) and ancestor masks of a tree of n nodes in order."""
    parents = [-1] + [i - 1 if chain else int(rng.integers(0, i)) for i in range(1, n)]
    masks = []
    for i in range(n):
        masks.append((1 << i) | (masks[parents[i]] if parents[i] >= 0 else 0))
    return parents[:n], masks[:n]


def visible(masks, n, L, window):
    """[n, L] truth: what each node attends to."""
    prefix = L - n
    keep = (1 << n) - 1
    own = [m & keep for m in masks]
    depth = [bin(m & ~(1 << i)).count("1") for i, m in enumerate(own)]
    vis = np.zeros((n, L), bool)
    for i in range(n):
        vis[i, :prefix] = True
        if window > 0:
            vis[i, :max(0, min(prefix, prefix + depth[i] - window + 1))] = False
        for j in range(n):
            if own[i] >> j & 1 and not (window > 0 and depth[i] - depth[j] >= window):
                vis[i, prefix + j] = True
    return vis


def tree_attention(q, keys, values, masks, L, scale, window):
    """One row.  q [n, Hq, D], keys / values [L, Hkv, D], all float64.  Returns out, lse, and per
    output what the bounds need: spread = sum_j p_j |v_j| and the largest sum_d |q_d k_d| * scale."""
    n, Hq, D = q.shape
    G = Hq // keys.shape[1]
    vis = visible(masks, n, L, window)
    out, spread = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, size = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for i in range(n):
        at = np.nonzero(vis[i])[0]
        if len(at) == 0:
            continue
        for h in range(Hq):
            k, v = keys[at, h // G], values[at, h // G]
            s = k @ q[i, h] * scale
            m = s.max()
            p = np.exp(s - m)
            out[i, h] = p @ v / p.sum()
            spread[i, h] = p @ np.abs(v) / p.sum()
            lse[i, h] = m + np.log(p.sum())
            size[i, h] = (np.abs(k) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, spread, size


def check_tree(got_o, got_l, out, lse, spread, size, D, lost=0.0):
    """The bounds: products of two 8-bit-significand values are exact in fp32 and a sum of D of them
    is off by at most D steps of 2^-23 of the sum of magnitudes, so a score by es = 2 (D + 16) 2^-23 size (two
    for the scaling and the exponential's own error); a weight by a factor e^es and, as a matrix operand,
    half a bf16 step (2^-8); their sum is normalised in fp32; the output is rounded once (2^-8).
    lost: what weights too small for their operand's type leave out (0 with bf16 operands)."""
    es = 2 * (D + 16) * 2.0 ** -23 * size + 2.0 ** -18
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * es[..., None]) * 1.01 * spread + lost + 1e-30
    err = np.abs(got_o - out)
    assert np.all(np.isfinite(got_o)), "not finite"
    worst = np.unravel_index(np.argmax(err / tol), err.shape)
    assert np.all(err <= tol), f"out off by {err[worst]:.3e} where {tol[worst]:.3e} is allowed, at {worst}"
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(got_l), empty)
    el = np.abs(np.where(empty, 0, got_l) - np.where(empty, 0, lse))
    tl = es + 2.0 ** -21 * np.abs(np.where(empty, 0, lse))
    assert np.all(el <= tl), f"lse off by {el.max():.3e}"


def plan(context_lens, new_lens, held, free_list, free_count, table, P, max_tokens, num_pages, parents=None):
    """The plan of a step, row after row, in plain Python integers."""
    B, W = table.shape
    table, free_list = table.copy(), list(free_list)
    bits, BAD_PAGE, BAD_LEN, NO_PAGES, BAD_TREE = 0, 1, 2, 0x10, 0x40
    lens_out, held_out = list(context_lens), list(held)
    start = [0]
    for n in new_lens:
        start.append(start[-1] + max(0, n))
    stack = free_list[:free_count]
    for b in range(B):
        if new_lens[b] < 0:
            if 0 <= held[b] <= W:
                stack += [int(x) for x in table[b, :held[b]]]
            else:
                bits |= BAD_LEN
            lens_out[b] = held_out[b] = 0
    free_list[free_count:len(stack)] = stack[free_count:]
    top, wanted, ok = len(stack), 0, [False] * B
    for b in range(B):
        n = new_lens[b]
        if n < 0:
            continue
        pages = -(-(context_lens[b] + n) // P)
        if context_lens[b] < 0 or not 0 <= held[b] <= W or pages > W or start[b] + n > max_tokens:
            bits |= BAD_LEN
            continue
        need = max(0, pages - held[b]) if n > 0 else 0
        wanted += need
        if need and wanted > top:
            bits |= NO_PAGES
            continue
        ok[b] = True
        for j in range(need):
            table[b, held[b] + j] = stack.pop()
        lens_out[b], held_out[b] = context_lens[b] + n, held[b] + need
    slots, pos, mask = [-1] * max_tokens, [0] * max_tokens, [0] * max_tokens
    for b in range(B):
        n, masks = start[b + 1] - start[b], []
        for i in range(n):
            t = start[b] + i
            if t >= max_tokens:
                break
            depth = i
            if parents is not None and n <= 64:
                p = int(parents[t])
                if p < -1 or p >= i:
                    bits, p = bits | BAD_TREE, -1
                masks.append((1 << i) | (masks[p] if p >= 0 else 0))
                mask[t] = masks[-1]
                depth = bin(masks[-1]).count("1") - 1
            pos[t] = context_lens[b] + depth
            if ok[b]:
                page = int(table[b, (context_lens[b] + i) // P])
                if 0 <= page < num_pages:
                    slots[t] = page * P + (context_lens[b] + i) % P
                else:
                    bits |= BAD_PAGE
    return dict(table=table, free_list=np.array(free_list), lens=lens_out, held=held_out, count=len(stack), start=start,
                slots=slots, positions=pos, mask=mask, bits=bits)


def norm_rope(x, weight, cos_sin, rot, interleaved, eps):
    """x [T, H, D] float64 (rows of cos_sin already picked: [T, rot])."""
    y = x.copy()
    if weight is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    c, s = cos_sin[:, None, :rot // 2], cos_sin[:, None, rot // 2:]
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    u, v = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return y
