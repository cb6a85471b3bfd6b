"""The tree-drafting operators where one row, node or token could reach into another's result, and at the ends
of their ranges."""
import math

import numpy as np
import pytest
import torch

import tree_refs as R
from test_tree_ops_gpu import (Tree, check_plan, compact_case, compacted, dev, f64, i32, pa, plan_case, raw,  # noqa: F401
                               rope_call, rope_case, stored_ok)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------ rows that a plan refuses

def test_plan_says_which_rows_it_granted(pa):
    """1: the row's tokens have their places (also where it has none); 0: refused, for whatever reason, or ended."""
    P = 16
    lens, news, held = [40, 3, 16, 5, -1, 20, 33, 100], [9, 2, 1, 0, 2, -1, 1, 1], [3, 1, 1, 1, 1, 2, 3, 7]
    #      ok: the page that row 5 gives back, ok, second page, nothing to do, bad length, ended, ok, over the tokens
    table = np.arange(8 * 7).reshape(8, 7)
    for in_place in (False, True):
        a = [i32(x) for x in (lens, news, held)] + [i32(list(range(60, 61)) + [0] * 60), i32([0]), i32(table)]
        out = {} if in_place else {k: i32([0] * n) for k, n in (("context_lens_out", 8), ("held_pages_out", 8), ("free_count_out", 1))}
        granted, st = i32([7] * 8), i32([0])
        pa.pa_plan_step(*a, i32([0] * 9), dev([0] * 15, torch.int64), i32([0] * 15), page_size=P, granted=granted,
                        status=st, **out)
        assert granted.tolist() == [1, 1, 1, 1, 0, 0, 1, 0], granted.tolist()
        assert int(st) == pa.PA_DEV_BAD_LEN
        a = [i32(x) for x in (lens, news, [1, 1, 1, 1, 1, 1, 3, 7])] + [i32([0] * 61), i32([0]), i32(table)]
        pa.pa_plan_step(*a, i32([0] * 9), dev([0] * 99, torch.int64), i32([0] * 99), page_size=P, granted=granted,
                        status=st, **out)
        # row 0 wants three pages, one is given back: it and row 2 get none, those that need none have their places
        assert granted.tolist() == [0, 1, 0, 1, 0, 0, 1, 1], granted.tolist()
        assert int(st) == pa.PA_DEV_BAD_LEN | pa.PA_DEV_NO_PAGES


def test_tree_leaves_refused_rows_alone(pa):
    rows = [(100, 4), (64, 9), (33, 33), (200, 6), (5, 5)]
    for fmt in ("bf16", "fp8", "nvfp4"):
        t = Tree(400, rows, 8, 2, 128, 16, fmt)
        args = list(t.args())
        args[4][1], args[4][4] = 3, -8  # lengths that would not do
        args[3][1, :] = 1 << 20         # and pages
        out = torch.full(t.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(t.q.shape[:2], 7.0, device="cuda")
        ws = pa.workspace_for_tree(t.q, t.k, args[3], 33)
        more = {} if fmt == "bf16" else {"k_scale": t.scales[0], "v_scale": t.scales[1]}
        fn = {"bf16": pa.pa_tree_gqa, "fp8": pa.pa_tree_gqa_fp8, "nvfp4": pa.pa_tree_gqa_nvfp4}[fmt]
        fn(*args, out, lse, max_query=33, scale=t.scale, workspace=ws, granted=i32([1, 0, 1, 1, 0]), **more)
        torch.cuda.synchronize()
        assert pa.pa_read_device_status(ws) == 0
        o, l, spread, size = t.reference()
        for b in (0, 2, 3):
            s = slice(int(t.start[b]), int(t.start[b + 1]))
            R.check_tree(f64(out[s]), f64(lse[s]), o[s], l[s], spread[s], size[s], t.D, t.lost())
        for b in (1, 4):
            s = slice(int(t.start[b]), int(t.start[b + 1]))
            assert bool((out[s] == 7.0).all()) and bool((lse[s] == 7.0).all())


def test_compact_leaves_refused_and_long_rows_alone(pa):
    rows = [(50, 9), (40, 9), (90, 70), (64, 64), (33, 5)]
    paths = [[0, 2, 8], [], [], list(range(1, 64)), []]
    for layers in (0, 3):
        c = compact_case(5, rows, layers, 2, 64, 16, torch.bfloat16, paths)
        want, lens = compacted(c)
        lens[1], lens[2], lens[4] = 40, 90, -6
        acc, num = c["acc"].copy(), list(c["num"])
        acc[1, :3], num[1] = [0, 2, 5], 3  # a path of nodes that are not in the cache
        acc[2, :3], num[2] = [3, 9, 60], 3
        acc[4, :2], num[4] = [9, 3], 99
        st, out = i32([0]), i32([-9] * 5)
        pa.pa_kv_compact(c["k"], c["v"], i32(c["table"]), i32([50, 40, 90, 64, -6]), i32(c["start"]), i32(acc), i32(num),
                         granted=i32([1, 0, 1, 1, 0]), context_lens_out=out, status=st)
        torch.cuda.synchronize()
        assert int(st) == 0 and out.tolist() == lens
        assert np.array_equal(raw(c["k"]), want[0]) and np.array_equal(raw(c["v"]), want[1])


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_steps_in_which_pages_run_out(pa, fmt, captured):
    """Plan, norm + rotation + write, attention and compaction, each on what the ones before left on the GPU, called one by one
    or replayed from a graph, with too few pages: granted rows' attention is that of the tokens that they hold; a refused row keeps its
    length, its tokens and their bytes, and no call says that anything but pages was missing."""
    rng, g = np.random.default_rng(21), torch.Generator().manual_seed(21)
    hq, hkv, D, P, pages, B, T, eps, M = 8, 2, 128, 16, 9, 5, 150, 1e-6, 14
    width, kind = (D, torch.bfloat16) if fmt == "bf16" else (R.row_bytes(fmt, D), torch.uint8)
    scales = {"bf16": (1.0, 1.0), "fp8": (0.013, 0.021), "nvfp4": (0.25, 0.25)}[fmt]
    sc = {} if fmt == "bf16" else dict(k_scale=scales[0], v_scale=scales[1])
    write = {"bf16": pa.pa_qk_norm_rope_write, "fp8": pa.pa_qk_norm_rope_write_fp8, "nvfp4": pa.pa_qk_norm_rope_write_nvfp4}[fmt]
    attend = {"bf16": pa.pa_tree_gqa, "fp8": pa.pa_tree_gqa_fp8, "nvfp4": pa.pa_tree_gqa_nvfp4}[fmt]
    kp, vp = (torch.zeros(pages, P, hkv, width, dtype=kind, device="cuda") for _ in range(2))
    angle = torch.rand(512, D // 2, generator=g, dtype=torch.float64) * 6.28
    cs = torch.cat((angle.cos(), angle.sin()), -1).float().cuda()
    wq, wk = (torch.randn(D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    z = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    lens, lens2, held, count, fl, table = z(B), z(B), z(B), i32([pages]), i32(rng.permutation(pages)), z(B, 20) - 1
    start, slots, pos, mask, granted = z(B + 1), z(T, d=torch.int64), z(T), z(T, d=torch.int64), z(B)
    q_out = z(T, hq, D, d=torch.bfloat16)
    out, lse = torch.zeros_like(q_out), z(T, hq, d=torch.float32)
    ws, st = pa.workspace_for_tree(q_out, kp, table, M), z(1)
    news_d, parents_d, paths_d, num_d = z(B), z(T), z(B, M), z(B)
    x = z(T, hq + 2 * hkv, D, d=torch.bfloat16)

    def step():
        pa.pa_plan_step(lens, news_d, held, fl, count, table, start, slots, pos, page_size=P, parents=parents_d, tree_mask=mask,
                        granted=granted, status=st)
        write(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], wq, wk, cs, pos, slots, q_out, kp, vp, eps=eps, status=st, **sc)
        attend(q_out, kp, vp, table, lens, start, mask, out, lse, max_query=M, scale=D ** -0.5, workspace=ws, granted=granted, **sc)
        pa.pa_kv_compact(kp, vp, table, lens, start, paths_d, num_d, granted=granted, context_lens_out=lens2, status=st)
        lens.copy_(lens2)

    graph = None
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()  # no new tokens: nothing changes but what is set up at a first call
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    kept = [[] for _ in range(B)]  # per row: (key bytes, value bytes) of its tokens
    refused = longest = long_rows = 0
    for k in range(14):
        news = [int(rng.integers(0, M + 1)) for _ in range(B)]
        if k == 6:
            news[int(np.argmax([len(r) for r in kept]))] = -1
        if k == 8:
            news = [0, -1, -1, -1, -1]
        if k == 9:  # prompts: more tokens than a tree has, kept as they are
            news = [3, 70, 2, 0, 66]
        trees = [R.random_tree(rng, n) if 0 < n <= 64 else ([-1] * max(n, 0), []) for n in news]
        parents = [p for tr in trees for p in tr[0]]
        path = [[i for i in range(n) if tr[1][n - 1] >> i & 1] if 0 < n <= 64 else [] for n, tr in zip(news, trees)]
        news_d.copy_(i32(news))
        parents_d.copy_(i32(parents + [-1] * (T - len(parents))))
        paths_d.copy_(i32([p + [0] * (M - len(p)) for p in path]))
        num_d.copy_(i32([len(p) for p in path]))
        x.copy_((torch.randn(T, hq + 2 * hkv, D, generator=g) * 2).to(torch.bfloat16))
        st.zero_()
        torch.cuda.synchronize()
        (graph.replay if graph else step)()
        torch.cuda.synchronize()
        ok, hs, hl, ht = granted.tolist(), start.tolist(), lens.tolist(), table.cpu().numpy()
        long_row = any(ok[b] and n > M for b, n in enumerate(news))
        long_rows += long_row
        assert int(st) & ~pa.PA_DEV_NO_PAGES == 0
        assert bool(int(st)) == any(n >= 0 and not ok[b] for b, n in enumerate(news))
        assert pa.pa_read_device_status(ws) == (pa.PA_DEV_BAD_LEN if long_row else 0)
        flat = [raw(p).reshape(-1, hkv, raw(p).shape[-1]) for p in (kp, vp)]
        hm = mask.cpu().numpy().view(np.uint64)
        ek = R.norm_rope(f64(x[:, hq:hq + hkv]), f64(wk), f64(cs)[pos.cpu().numpy()], D, False, eps)
        ev = f64(x[:, hq + hkv:])
        for b, n in enumerate(news):
            held_bytes = [tuple(f[int(ht[b, i // P]) * P + i % P] for f in flat) for i in range(hl[b])]
            if n < 0:
                assert hl[b] == 0 and ok[b] == 0
                kept[b] = []
                continue
            refused += not ok[b]
            take = list(range(n)) if n > 64 else path[b]
            assert hl[b] == len(kept[b]) + (len(take) if ok[b] else 0)
            for mine, then in zip(held_bytes, kept[b]):
                assert np.array_equal(mine[0], then[0]) and np.array_equal(mine[1], then[1])
            if not ok[b] or n == 0:
                continue
            for (kk, vv), i in zip(held_bytes[len(kept[b]):], take):
                assert np.all(stored_ok(kk, ek[hs[b] + i], fmt, D, scales[0])) and np.all(stored_ok(vv, ev[hs[b] + i], fmt, D, scales[1]))
            if n <= 64:  # the nodes of the accepted path attend to what the row now holds, in order
                at = [hs[b] + i for i in path[b]]
                keys, vals = (R.pool_values(np.stack([r[w] for r in held_bytes]), fmt, D, scales[w]) for w in (0, 1))
                chain = [(2 << i) - 1 for i in range(len(at))]
                ref = R.tree_attention(f64(q_out[at]), keys, vals, chain, hl[b], D ** -0.5, 0)
                lost = 0.0 if fmt == "bf16" else 2.0 ** -32 * hl[b] * float(np.abs(vals).max())
                R.check_tree(f64(out[at]), f64(lse[at]), *ref, D, lost)
            kept[b] = held_bytes
            longest = max(longest, hl[b])
    assert refused >= 5 and longest >= 40 and long_rows


# ------------------------------------------------------------------------------------------ tree attention

@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 128), (8, 2, 256), (6, 3, 64), (64, 2, 128)])
def test_tree_large_keys_of_other_nodes(pa, fmt, hq, hkv, D):
    """A node's key that raises its own running maximum far changes no bit of the nodes that do not attend to it."""
    rows, G, j = [(700, 13), (1033, 20)], hq // hkv, 5
    masks = [1 | 1 << i for _, n in rows for i in range(n)]  # all nodes are children of the first
    t = Tree(300 + D, rows, hq, hkv, D, 16, fmt, masks=masks)
    want, want_l, _ = t.call(pa, num_splits=1)
    for b, (L, n) in enumerate(rows):
        tok = L - n + j
        row = t.k[int(t.table[b, tok // 16]), tok % 16]
        for g in range(hkv):
            up = t.q[int(t.start[b]) + j, g * G].float() > 0  # large scores in the node's own first head
            if fmt == "bf16":
                row[g] = torch.where(up, 50.0, -50.0).to(torch.bfloat16)
            elif fmt == "fp8":
                row[g] = torch.where(up, 0x7E, 0xFE).to(torch.uint8)
            else:
                code = torch.where(up, 7, 15)
                row[g, :D // 2] = (code[::2] | code[1::2] << 4).to(torch.uint8)
                row[g, D // 2:D // 2 + D // 16] = 0x70
    out, lse, ws = t.call(pa, num_splits=1)
    torch.cuda.synchronize()
    assert pa.pa_read_device_status(ws) == 0
    others = [int(t.start[b]) + i for b, (_, n) in enumerate(rows) for i in range(n) if i != j]
    assert not torch.equal(lse[int(t.start[0]) + j], want_l[int(t.start[0]) + j])
    assert torch.equal(lse[others], want_l[others]) and torch.equal(out[others], want[others])


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("exponent", [117, -116])
def test_tree_queries_near_the_ends_of_their_range(pa, fmt, exponent):
    """Queries of 2^119 or 2^-116 under a scale that brings the scores back to tens."""
    t = Tree(310, [(300, 9), (64, 20), (1, 1)], 8, 2, 128, 16, fmt, big_q=2.0 ** exponent)
    t.scale = 2.0 ** (4 - exponent) / math.sqrt(128)
    t.check(pa)


# ------------------------------------------------------------------------------------------ plan

@pytest.mark.parametrize("free", [6, 2, 1])
def test_plan_rows_whose_pages_do_not_hold_their_context(pa, free):
    """The pages that a row needs are those of its context and its new tokens, less the held ones, with or without
    new tokens."""
    P, W = 16, 6
    lens, news, held = [40, 5, 33, 20], [0, 3, 2, 0], [1, 0, 3, 2]
    need = [max(0, -(-(n + k) // P) - h) for n, k, h in zip(lens, news, held)]
    assert need == [2, 1, 0, 0]
    table = np.full((4, W), -1)
    table[0, 0], table[2, :3], table[3, :2] = 10, [11, 12, 13], [14, 15]
    want_t, want_l, want_h, stack, wanted, refused = table.copy(), list(lens), list(held), list(range(free)), 0, []
    for b in range(4):
        wanted += need[b]
        if need[b] and wanted > free:
            refused.append(b)
            continue
        for x in range(need[b]):
            want_t[b, held[b] + x] = stack.pop()
        want_l[b], want_h[b] = lens[b] + news[b], held[b] + need[b]
    for in_place in (False, True):
        tl, tn, th, tt, tf, tc = i32(lens), i32(news), i32(held), i32(table), i32(list(range(free)) + [0] * (16 - free)), i32([free])
        out = {} if in_place else dict(context_lens_out=torch.empty_like(tl), held_pages_out=torch.empty_like(th),
                                       free_count_out=torch.empty_like(tc))
        start, slots, pos, st = i32([0] * 5), dev([0] * 8, torch.int64), i32([0] * 8), i32([0])
        pa.pa_plan_step(tl, tn, th, tf, tc, tt, start, slots, pos, page_size=P, status=st, **out)
        got = (tl, th, tc) if in_place else tuple(out.values())
        assert got[0].tolist() == want_l and got[1].tolist() == want_h and int(got[2]) == len(stack)
        assert np.array_equal(tt.cpu().numpy(), want_t) and start.tolist() == [0, 0, 3, 5, 5]
        assert int(st) == (pa.PA_DEV_NO_PAGES if refused else 0)
        row1 = [-1] * 3 if 1 in refused else [int(want_t[1, 0]) * P + 5 + i for i in range(3)]
        assert slots.tolist() == row1 + [13 * P + 1, 13 * P + 2] + [-1] * 3



@pytest.mark.parametrize("tokens", [0, 3, 5000])
@pytest.mark.parametrize("B", [1708, 8192])
def test_plan_most_rows(pa, B, tokens):
    """As many rows as there may be, in one cluster, apart and with the state in a launch of its own; no tokens at all."""
    c = plan_case(B + tokens, B, 16, 60, 1, ended=B // 9)
    c["news"] = [n if n < 0 or b % 3 == 0 and b < 3 * tokens else 0 for b, n in enumerate(c["news"])]
    check_plan(pa, c, max_tokens=tokens)
    c["news"][5] = 2  # one token too many, or two
    check_plan(pa, c, max_tokens=sum(max(0, n) for n in c["news"]) - 1)


# ------------------------------------------------------------------------------------------ norm, rotation, write

@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("hq,hkv,D", [(4, 1, 128), (3, 2, 128), (4, 1, 64), (5, 2, 64), (2, 1, 256), (4, 2, 128)])
@pytest.mark.parametrize("scale", [0.013, 0.021, 0.3, 0.7, 0.25])
def test_rope_write_values_are_the_plain_write(pa, fmt, hq, hkv, D, scale):
    """Whichever rows a value's row shares a warp with, its codes are pa_kv_write's: zeros of either sign, infinities and NaN
    among them."""
    c = rope_case(20 + hq + D, 40, hq, hkv, D, D, fmt=fmt, pad=3)
    c["scales"] = (scale, scale)
    c["v"][:, :, ::7] = -0.0
    c["v"][1, 0, 3], c["v"][2, 0, 5], c["v"][3, 0, 9], c["v"][4, 0, 0] = math.inf, -math.inf, math.nan, 0.0
    c["v"][5] *= 1e30
    c["v"][6] *= 1e-30
    kp, vp = c["kp"].clone(), c["vp"].clone()
    fn = {"fp8": pa.pa_kv_write_fp8, "nvfp4": pa.pa_kv_write_nvfp4}[fmt]
    fn(c["k"].contiguous(), c["v"].contiguous(), c["slots"], kp, vp, k_scale=scale, v_scale=scale)
    for interleaved in (False, True):
        rope_call(pa, c, interleaved=interleaved)
        assert np.array_equal(raw(c["vp"]), raw(vp))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv,D", [(4, 2, 128), (3, 1, 64), (2, 1, 256), (4, 1, 128)])
def test_rope_write_nvfp4_keys_without_turn_are_the_plain_write(pa, hq, hkv, D, interleaved):
    """Block scales and padding byte for byte; codes too, but for the sign of a zero (x cos - y sin loses it)."""
    c = rope_case(40 + D, 60, hq, hkv, D, D, fmt="nvfp4", pad=4)
    c["cos_sin"] = torch.cat((torch.ones(c["far"], D // 2), torch.zeros(c["far"], D // 2)), -1).cuda()
    c["k"][3, 0, :40] = 0.0
    c["k"][4] *= 1e4  # block scales past 448
    c["k"][5] *= 1e-5
    kp, vp = c["kp"].clone(), c["vp"].clone()
    pa.pa_kv_write_nvfp4(c["k"].contiguous(), c["v"].contiguous(), c["slots"], kp, vp, **dict(zip(("k_scale", "v_scale"), c["scales"])))
    rope_call(pa, c, None, None, interleaved)
    mine, theirs = raw(c["kp"]), raw(kp)
    assert np.array_equal(mine[..., D // 2:], theirs[..., D // 2:])
    for nibble in (mine[..., :D // 2] & 15, theirs[..., :D // 2] & 15), (mine[..., :D // 2] >> 4, theirs[..., :D // 2] >> 4):
        assert np.all((nibble[0] == nibble[1]) | ((nibble[0] | nibble[1]) & 7 == 0))


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("hq,hkv,D,rot,interleaved", [(4, 2, 128, 128, False), (4, 1, 64, 32, False), (2, 2, 256, 128, True),
                                                     (3, 1, 128, 128, True)])
def test_rope_write_key_codes_are_nearest(pa, fmt, hq, hkv, D, rot, interleaved):
    """Normed and rotated keys: each code is the one nearest to the quotient in 64 bits, within the arithmetic before it.  The sum
    of squares has at most 11 roundings of 2^-24 (a lane's four products and one sum, five exchanges, + eps), of which the root
    takes half; the product with the weight is exact, u cos - v sin rounded once, the last product once: 7.5 x 2^-24 of the
    quotient, less than 2^-21."""
    c = rope_case(60 + D, 2000, hq, hkv, D, rot, fmt=fmt)
    rope_call(pa, c, interleaved=interleaved)
    cs = f64(c["cos_sin"])[c["positions"].cpu().numpy()]
    x = R.norm_rope(f64(c["k"]), f64(c["wk"]), cs, rot, interleaved, 1e-6) / float(np.float32(c["scales"][0]))
    got = raw(c["kp"]).reshape(-1, hkv, c["kp"].shape[-1])[c["slots"].cpu().numpy()]
    off = 2.0 ** -21
    near = np.sort(R.e4m3_table()[:127])

    def nearest(values, at, err, codes):
        """values are among `codes` (ascending, >= 0) the nearest to |at|, if |at| is off by at most err."""
        mid = (codes[1:] + codes[:-1]) / 2
        lo, hi = np.searchsorted(mid, np.abs(at) - err, "left"), np.searchsorted(mid, np.abs(at) + err, "right")
        mine = np.searchsorted(codes, np.abs(values))
        return (codes[np.minimum(mine, len(codes) - 1)] == np.abs(values)) & (lo <= mine) & (mine <= hi)

    if fmt == "fp8":
        assert nearest(R.e4m3_table()[got], x, off * np.abs(x), near).all()
        return
    blk = R.e4m3_table()[got[..., D // 2:D // 2 + D // 16]]
    amax = np.abs(x).reshape(*x.shape[:-1], D // 16, 16).max(-1) / 6
    assert nearest(blk, amax, off * 1.5 * amax, near).all()  # (and the division by 6)
    by = np.repeat(blk, 16, -1)
    val = R.pool_values(got, "nvfp4", D, 1.0)
    assert (val[by == 0] == 0).all()
    some = by > 0
    y = x[some] / by[some]
    assert nearest(val[some] / by[some], y, off * 1.5 * np.abs(y), R.E2M1).all()
