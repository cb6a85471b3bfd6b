"""Plain references (numpy, 64 bits) of the streams' operators.  Test infrastructure; shares no code with the library."""
from __future__ import annotations

import numpy as np


def visible(L, n, window, first):
    """[n, L] truth: what each of the row's n newest tokens attends to."""
    p = np.arange(L - n, L)[:, None]
    t = np.arange(L)
    v = t <= p
    if window > 0:
        v &= (t > p - window) | (t < first)
    return v


def stream_attention(q, keys, values, L, scale, window, first):
    """One row.  q [n, Hq, D], keys / values [L, Hkv, D] in 64 bits (what nobody sees may be anything).  Returns out, lse, and per output what
    the bounds need: spread = sum_j p_j |v_j| and the largest sum_d |q_d k_d| * scale."""
    n, Hq, D = q.shape
    G = Hq // keys.shape[1]
    vis = visible(L, n, window, first)
    at = np.nonzero(vis.any(0))[0]  # (the others' keys may be no numbers)
    vis = vis[:, at]
    out, spread = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, size = np.zeros((n, Hq)), np.zeros((n, Hq))
    for h in range(Hq):
        k, v = keys[at, h // G], values[at, h // G]
        s = np.where(vis, q[:, h] @ k.T * scale, -np.inf)
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        Z = p.sum(1, keepdims=True)
        out[:, h], spread[:, h] = p @ v / Z, p @ np.abs(v) / Z
        lse[:, h] = m[:, 0] + np.log(Z[:, 0])
        size[:, h] = np.where(vis, np.abs(q[:, h]) @ np.abs(k).T, 0).max(1) * abs(scale)
    return out, lse, spread, size


def release(lens, held, start, free_list, free_count, table, P, num_pages, window, first, ended=None):
    """The release of a step's pages, row after row, in plain Python integers."""
    B, W = table.shape
    table, stack, bits, F = table.copy(), [int(x) for x in free_list[:max(0, min(free_count, num_pages))]], 0, -(-first // P)
    if len(stack) != free_count:
        bits |= 2
    lens_out, held_out, start_out = list(lens), list(held), list(start)
    for b in range(B):
        if lens[b] < 0 or not 0 <= held[b] <= W or not 0 <= start[b] <= held[b]:
            bits |= 2
            continue
        if ended is not None and ended[b]:
            pages = [j for j in range(held[b]) if not F <= j < start[b]]
            lens_out[b] = held_out[b] = start_out[b] = 0
        else:
            behind = min(max(0, lens[b] + 1 - window) // P, held[b])
            pages = [j for j in range(behind) if j >= F and j >= start[b]]
            if pages:
                start_out[b] = behind
            elif behind > F:
                start_out[b] = max(start[b], behind)
        for j in pages:
            page = int(table[b, j])
            if not 0 <= page < num_pages:
                bits |= 1
            if len(stack) < num_pages:
                stack.append(page)
            else:
                bits |= 2
            table[b, j] = -1
    free = list(free_list)
    free[:len(stack)] = stack
    return dict(table=table, free_list=np.array(free), count=len(stack), lens=lens_out, held=held_out, start=start_out, bits=bits)
