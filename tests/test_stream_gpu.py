"""The streams' operators on the GPU against plain references in 64 bits: attention of single tokens, chunks and prompts in a
window beside the first tokens, pages released behind the window, and steps of them together."""
import math

import numpy as np
import pytest
import torch

import stream_refs as S
import tree_refs as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_attention_19_gb300 as pkg
    return pkg


def dev(a, dtype=None):
    return torch.as_tensor(np.asarray(a)).to("cuda", dtype)


def i32(a):
    return dev(np.asarray(a, np.int64), torch.int32)


def raw(t):
    return (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).cpu().numpy().view(
        np.uint16 if t.dtype == torch.bfloat16 else np.uint8)


def f64(t):
    return t.double().cpu().numpy()


NAN_BYTE = 0x7F


class Rows:
    """Rows of (L, n) over a shuffled pool; slots that no row fills, and pages that nobody sees, hold NaN, and the table
    has no page for the latter."""

    def __init__(self, seed, rows, hq, hkv, D, page, fmt="bf16", window=0, first=0, extra=3, shuffle=True, big_q=1.0,
                 offset=0):
        rng = np.random.default_rng(seed)
        self.rows, self.hq, self.hkv, self.D, self.page, self.fmt = rows, hq, hkv, D, page, fmt
        self.window, self.first = window, first
        g = torch.Generator().manual_seed(seed)
        pages = [-(-L // page) for L, _ in rows]
        total = sum(pages) + 2
        order = rng.permutation(total)
        order = (order if shuffle else np.arange(total)) + offset
        W = max(pages + [1]) + 1
        self.table = np.full((len(rows), W), -7, np.int64)  # entries behind a row's last page are not read
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.scales = {"bf16": (1.0, 1.0), "fp8": (0.013, 0.021), "nvfp4": (0.25, 0.0625)}[fmt]
        width = D if fmt == "bf16" else R.row_bytes(fmt, D)
        pools = []
        for _ in range(2):
            if fmt == "bf16":
                p = torch.full((total, page, hkv, D), math.nan).to(torch.bfloat16)
            else:
                p = torch.full((total, page, hkv, width), NAN_BYTE, dtype=torch.uint8)
            pools.append(p)
        for b, (L, n) in enumerate(rows):
            if L == 0:
                continue
            t = np.arange(L)
            pg, off = self.table[b, t // page] - offset, t % page
            for p in pools:
                x = torch.randn(L, hkv, D, generator=g)
                if fmt == "bf16":
                    v = x.to(torch.bfloat16)
                elif fmt == "fp8":
                    v = (x / 0.015).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                else:
                    v = torch.zeros(L, hkv, width, dtype=torch.uint8)
                    v[..., :D // 2] = torch.randint(0, 256, (L, hkv, D // 2), generator=g).to(torch.uint8)
                    blk = (torch.rand(L, hkv, D // 16, generator=g) * 2 + 0.25).to(torch.float8_e4m3fn)
                    v[..., D // 2:D // 2 + D // 16] = blk.view(torch.uint8)
                if n > 0:
                    hidden = ~S.visible(L, n, window, first).any(0)
                    v[torch.as_tensor(hidden)] = math.nan if fmt == "bf16" else NAN_BYTE
                p[pg, off] = v
            if n > 0 and window > 0:
                for j in range(-(-first // page), max(0, L - n + 1 - window) // page):
                    self.table[b, j] = -1
        self.offset = offset
        if offset:
            self.k, self.v = (torch.empty(total + offset, page, hkv, p.shape[-1], dtype=p.dtype, device="cuda") for p in pools)
            self.k[offset:], self.v[offset:] = pools[0].cuda(), pools[1].cuda()
        else:
            self.k, self.v = (p.cuda() for p in pools)
        self.start = np.concatenate(([0], np.cumsum([n for _, n in rows]))).astype(int)
        self.T = int(self.start[-1])
        self.extra = extra  # padded tokens behind the last row
        self.q = (torch.randn(self.T + extra, hq, D, generator=g) * big_q).to(torch.bfloat16).cuda()
        self.scale = 1.0 / math.sqrt(D)

    def args(self):
        return (self.q, self.k, self.v, i32(self.table), i32([L for L, _ in self.rows]), i32(self.start))

    def call(self, pa, max_query=None, num_splits=0, args=None, out=None, lse=None, ws=None, stream=None, granted=None):
        args = args or self.args()
        if out is None:
            out = torch.full(self.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
            lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        mq = max_query or max([n for _, n in self.rows] + [1])
        if ws is None:
            ws = pa.workspace_for_stream(self.q, self.k, args[3], mq, num_splits)
        fn = {"bf16": pa.pa_stream_gqa, "fp8": pa.pa_stream_gqa_fp8, "nvfp4": pa.pa_stream_gqa_nvfp4}[self.fmt]
        more = {} if self.fmt == "bf16" else {"k_scale": self.scales[0], "v_scale": self.scales[1]}
        fn(*args, out, lse, max_query=mq, scale=self.scale, window=self.window, first=self.first, num_splits=num_splits,
           workspace=ws, stream=stream, granted=granted, **more)
        return out, lse, ws

    def reference(self):
        k, v = self.k[self.offset:], self.v[self.offset:]
        kk, vv = R.pool_values(raw(k), self.fmt, self.D, self.scales[0]), R.pool_values(raw(v), self.fmt, self.D, self.scales[1])
        q, parts = f64(self.q), []
        for b, (L, n) in enumerate(self.rows):
            if n == 0:
                continue
            t = np.arange(L)
            pg, off = np.maximum(self.table[b, t // self.page] - self.offset, 0), t % self.page
            parts.append(S.stream_attention(q[self.start[b]:self.start[b + 1]], kk[pg, off], vv[pg, off], L, self.scale,
                                            self.window, self.first))
        return [np.concatenate(x) for x in zip(*parts)]

    def lost(self):
        """f16 weights (8- and 4-bit pools): a weight below 2^-14 is off by at most half of f16's smallest step, 2^-25.
        The largest weight of a row is at least 2^7, so their sum is too, and an output sum(w v) / sum(w) is off by at
        most 2^-25 / 2^7 sum(|v|) = 2^-32 sum(|v|) <= 2^-32 L max |v|.  bf16 weights have fp32's range: nothing."""
        if self.fmt == "bf16":
            return 0.0
        v = R.pool_values(raw(self.v[self.offset:]), self.fmt, self.D, self.scales[1])
        return 2.0 ** -32 * max(L for L, _ in self.rows) * float(np.nanmax(np.abs(v)))

    def check(self, pa, num_splits=0, max_query=None, **kw):
        out, lse, ws = self.call(pa, num_splits=num_splits, max_query=max_query, **kw)
        torch.cuda.synchronize()
        assert pa.pa_read_device_status(ws) == 0
        assert bool((out[self.T:] == 7.0).all()) and bool((lse[self.T:] == 7.0).all()), "tokens behind the last row"
        self.compare(out, lse)
        return out, lse

    def compare(self, out, lse):
        R.check_tree(f64(out[:self.T]), f64(lse[:self.T]), *self.reference(), self.D, self.lost())


LADDER = [(1, 1), (2, 2), (3, 1), (31, 7), (32, 5), (33, 33), (64, 16), (100, 0), (129, 12), (685, 20), (1000, 3), (200, 200),
          (131, 130), (515, 257)]
SHAPES = [(8, 2, 128, 16), (5, 5, 64, 32), (16, 2, 256, 32), (36, 3, 128, 8), (14, 2, 64, 128), (40, 2, 128, 64),
          (2, 2, 128, 256), (128, 1, 128, 16), (12, 4, 256, 8)]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("hq,hkv,D,page", SHAPES)
def test_stream_ladder(pa, fmt, hq, hkv, D, page):
    Rows(10 + hq + D, LADDER, hq, hkv, D, page, fmt).check(pa)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("hq,hkv,D,page", [(8, 2, 128, 16), (2, 2, 64, 8), (6, 1, 256, 32), (4, 4, 128, 64)])
@pytest.mark.parametrize("window,first", [(1, 0), (1, 1), (2, 5), (7, 64), (64, 4), (100, 16), (100, 17), (640, 130),
                                          (129, 1000), (5, 90), (100000, 3)])
def test_stream_window_and_first(pa, fmt, hq, hkv, D, page, window, first):
    Rows(50 + window + first, LADDER, hq, hkv, D, page, fmt, window, first).check(pa)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_stream_single_tokens(pa, fmt):
    rows = [(L, 1) for L in (1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000, 4097, 9001)]
    for window, first in ((0, 0), (64, 4), (1000, 33), (9, 0)):
        Rows(60 + window, rows, 16, 2, 128, 16, fmt, window, first).check(pa)
        Rows(61 + window, rows, 4, 4, 64, 32, fmt, window, first).check(pa)
        Rows(62 + window, rows, 8, 2, 256, 64, fmt, window, first).check(pa, max_query=1)


@pytest.mark.parametrize("splits", [1, 3, 64, 1000, 4096])
def test_stream_splits(pa, splits):
    rows = [(5000, 12), (3, 2), (900, 400), (1, 1), (77, 0), (2500, 1)]
    Rows(70, rows, 16, 2, 128, 16).check(pa, num_splits=splits)
    Rows(71, rows, 16, 2, 128, 16, "fp8", 300, 20).check(pa, num_splits=splits)
    Rows(72, rows, 4, 2, 256, 16, "bf16", 300, 20).check(pa, num_splits=splits)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("hq,hkv,D,n", [(8, 2, 128, 1), (8, 2, 128, 64), (2, 2, 64, 250), (8, 4, 256, 60)])
def test_stream_long_pieces_repeat(pa, fmt, hq, hkv, D, n):
    """Pieces of a hundred stages, of one tile and of two: the same bits twenty times, with a second call beside them."""
    t = Rows(110 + n, [(12900, n), (13001, n)], hq, hkv, D, 64, fmt)
    out, lse = t.check(pa, num_splits=4)
    other, side = Rows(111, [(3000, 40)], hq, hkv, D, 64, fmt), torch.cuda.Stream()
    args, pre = t.args(), (torch.zeros_like(out), torch.zeros_like(lse))
    ws, ws_other, args_other = pa.workspace_for_stream(t.q, t.k, args[3], n, 4), None, other.args()
    torch.cuda.synchronize()
    for _ in range(20):
        _, _, ws_other = other.call(pa, args=args_other, ws=ws_other, stream=side)
        t.call(pa, num_splits=4, args=args, out=pre[0], lse=pre[1], ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(pre[0][:t.T], out[:t.T]) and torch.equal(pre[1][:t.T], lse[:t.T])


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("rows,hkv", [([(700, 1)], 1), ([(300, 2), (650, 90)], 2), ([(513, 1)] * 3, 4)])
def test_stream_splits_cut_short_rows(pa, fmt, rows, hkv):
    """A number of shares that the caller gives holds for short rows too: their sums are then formed in parts, whose rounding shows
    in the log-sum-exps of hundreds of values."""
    t = Rows(112, rows, 64 * hkv, hkv, 64, 16, fmt)
    whole, parts = t.check(pa, num_splits=hkv), t.check(pa, num_splits=9 * hkv)
    assert not torch.equal(whole[1], parts[1])
    again = t.call(pa, num_splits=9 * hkv)
    assert torch.equal(again[0], parts[0]) and torch.equal(again[1], parts[1])


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
def test_stream_long(pa, fmt):
    Rows(73, [(20011, 6), (9000, 700), (3000, 3000)], 4, 1, 128, 64, fmt).check(pa)
    Rows(74, [(20011, 600), (9000, 1)], 4, 1, 64, 16, fmt, 2000, 100).check(pa)


@pytest.mark.parametrize("fmt,hq,hkv,D", [("bf16", 40, 40, 64), ("bf16", 66, 33, 128), ("fp8", 41, 41, 128), ("nvfp4", 90, 45, 64),
                                          ("bf16", 37, 37, 256), ("bf16", 160, 160, 64)])
def test_stream_many_key_heads(pa, fmt, hq, hkv, D):
    """More key heads than a group of CTAs has members: a CTA's share of the work holds several, and more than there are CTAs."""
    rows = [(200, 200), (3, 2), (700, 1), (150, 131), (64, 0)]
    Rows(100 + hkv, rows, hq, hkv, D, 16, fmt).check(pa)
    Rows(101 + hkv, rows, hq, hkv, D, 16, fmt, 60, 20).check(pa)
    Rows(102 + hkv, rows[:3], hq, hkv, D, 16, fmt, 60, 20).check(pa, num_splits=7)


@pytest.mark.parametrize("seed", range(30))
def test_stream_drawn(pa, seed):
    """Sizes, windows, formats and splits drawn over their whole ranges."""
    rng = np.random.default_rng(1000 + seed)
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    D, fmt = int(rng.choice([64, 128, 256])), str(rng.choice(["bf16", "fp8", "nvfp4"]))
    hkv, G = int(rng.choice([1, 2, 3, 5, 8, 19])), log(1, 128 if seed % 5 == 0 else 16)
    rows = []
    for _ in range(log(1, 40)):
        L = log(1, 3000 // hkv)
        rows.append((L, min(L, int(rng.choice([0, 1, 1, log(1, 40), log(1, max(1, 3000 // (G * hkv)))])))))
    window = int(rng.choice([0, log(1, 2000)]))
    Rows(200 + seed, rows, hkv * G, hkv, D, int(rng.choice([8, 16, 32, 64, 128, 256])), fmt, window,
         int(rng.choice([0, log(1, 300)])) if window else 0).check(pa, num_splits=int(rng.choice([0, 0, log(1, 300)])))


MIXED = [([16, 29, 4, 168, 126, 52, 3153, 70, 7, 12, 94, 2352, 6, 729, 226, 406, 303, 5, 977, 544, 9, 1309, 39, 3, 1755, 2, 22, 5],
          [0, 1, 12, 16, 35, 36, 49, 50, 51, 58, 66, 82, 124, 130, 131, 132, 133, 155, 156, 186, 212, 213, 248, 249, 250, 251, 252, 262, 267],
          56, 8, 128, 8, 2447, 4),
         ([80, 42, 53, 84, 72, 45, 40, 614, 88, 60, 78, 47, 61, 1424, 74, 76, 54, 114, 86, 50, 51, 3301, 46, 65, 70, 55, 43, 57, 265, 91, 63, 44, 66],
          [0, 1, 2, 3, 4, 5, 6, 7, 621, 622, 623, 624, 625, 626, 2050, 2051, 2052, 2053, 2167, 2168, 2169, 2170, 5471, 5472, 5473, 5474, 5475, 5476,
           5477, 5742, 5743, 5744, 5745, 5746], 64, 8, 64, 16, 18, 4)]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("lens,start,hq,hkv,D,page,window,first", MIXED)
def test_stream_mixed_tiles(pa, fmt, lens, start, hq, hkv, D, page, window, first):
    """Pieces of one tile, whose stages the two groups share, and of two, which take turns, in one CTA one after the other: the
    same bits ten times, and no wait that gives up."""
    rows = [(L, b - a) for L, a, b in zip(lens, start, start[1:])]
    t = Rows(150, rows, hq, hkv, D, page, fmt, window, first)
    out, lse, ws = t.call(pa)
    t.compare(out, lse)
    for _ in range(10):
        o, l, _ = t.call(pa, ws=ws)
        torch.cuda.synchronize()
        assert pa.pa_read_device_status(ws) == 0 and torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("window,first", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1), (300, 2 ** 31 - 1),
                                          (1, 2 ** 30), (0, 2 ** 31 - 1)])
@pytest.mark.parametrize("rows", [[(300, 1), (40, 1)], [(700, 300), (513, 2)]])
def test_stream_largest_windows_and_firsts(pa, fmt, window, first, rows):
    Rows(97, rows, 8, 2, 128, 16, fmt, window, first).check(pa)


def test_stream_many_rows(pa):
    """More rows than threads of a block, and than a wave of them."""
    Rows(75, [(1 + (i * 7) % 50, 1 if i % 9 else (i * 7) % 50 % 5) for i in range(2000)], 4, 2, 64, 8).check(pa)
    Rows(76, [(1 + (i * 7) % 300, 1 + (i * 5) % min(40, 1 + (i * 7) % 300)) for i in range(500)], 6, 2, 128, 16, "bf16", 50, 3).check(pa)


def test_stream_bound_of_queries_above_the_rows(pa):
    """max_query is a bound: the same results within rounding whatever tiles it chooses."""
    t = Rows(77, [(300, 3), (90, 1), (40, 17)], 8, 2, 128, 16, "bf16", 64, 9)
    for mq in (17, 32, 64, 65, 1000, 1 << 30):
        t.check(pa, max_query=mq)


def test_stream_no_row_has_a_query(pa):
    t = Rows(78, [(300, 0), (90, 0)], 8, 2, 128, 16)
    out, lse, ws = t.call(pa, max_query=4)
    torch.cuda.synchronize()
    assert pa.pa_read_device_status(ws) == 0 and bool((out == 7.0).all()) and bool((lse == 7.0).all())


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("hq,hkv,D,window,first", [(8, 2, 128, 0, 0), (8, 2, 128, 40, 10), (2, 2, 64, 90, 3), (1, 1, 128, 200, 0),
                                                   (8, 2, 256, 70, 20)])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_stream_tokens_do_not_see_others(pa, fmt, hq, hkv, D, window, first, what):
    """NaN (and infinite) keys and values of tokens that a token does not attend to change nothing of it; of tokens that it
    does, they reach it."""
    if what == "inf" and fmt != "bf16":
        pytest.skip("the 8- and 4-bit formats have no infinities")
    rows = [(350, 211), (30, 30), (164, 20), (300, 300)]
    t = Rows(80, rows, hq, hkv, D, 16, fmt, window, first)
    want, want_l, _ = t.call(pa)
    bad = []  # the row's last token, one in its middle and, under a window, its first new one; of the whole prompt a first token
    for b, (L, n) in enumerate(rows):
        for tok in {L - 1, L - n // 2} | ({L - n} if window > 0 and n < L else set()) | ({max(0, first - 1)} if n == 300 and first else set()):
            bad.append((b, tok))
            pg, off = int(t.table[b, tok // 16]), tok % 16
            for p in (t.k, t.v):
                if fmt == "bf16":
                    p[pg, off, :, ::3] = math.nan if what == "nan" else math.inf
                    if what == "inf":
                        p[pg, off, :, 1::3] = -math.inf
                else:
                    p[pg, off, :, -(t.k.shape[-1] // 4):] = NAN_BYTE
                    p[pg, off, :, t.D // 2:t.D // 2 + 4] = NAN_BYTE
    out, lse, ws = t.call(pa)
    torch.cuda.synchronize()
    seen = np.zeros(t.T, bool)
    for b, tok in bad:
        L, n = rows[b]
        seen[t.start[b]:t.start[b + 1]] |= S.visible(L, n, window, first)[:, tok]
    assert bool(seen.any()) and not bool(seen.all())
    clean = torch.as_tensor(np.nonzero(~seen)[0]).cuda()
    assert torch.equal(out[clean], want[clean]) and torch.equal(lse[clean], want_l[clean])
    hit = out[torch.as_tensor(np.nonzero(seen)[0]).cuda()].float()
    assert bool((~torch.isfinite(hit)).any(-1).all()), "a token that attends to such a token has no finite output"


@pytest.mark.parametrize("n,window,first", [(6, 0, 0), (200, 0, 0), (200, 50, 4)])
def test_stream_infinite_values_only(pa, n, window, first):
    """An infinite value with ordinary keys: the attending tokens get that infinity there, and finite results elsewhere; the others
    are as before."""
    rows = [(300, n)]
    t = Rows(81, rows, 4, 1, 64, 8, "bf16", window, first)
    want, want_l, _ = t.call(pa)
    tok = 300 - n + 3
    t.v[int(t.table[0, tok // 8]), tok % 8, 0, 5] = math.inf
    t.v[int(t.table[0, tok // 8]), tok % 8, 0, 9] = -math.inf
    out, lse, _ = t.call(pa)
    see = torch.as_tensor(S.visible(300, n, window, first)[:, tok]).cuda()
    assert torch.equal(out[:n][~see], want[:n][~see]) and torch.equal(lse, want_l)
    assert bool((out[:n][see][:, :, 5] == math.inf).all()) and bool((out[:n][see][:, :, 9] == -math.inf).all())
    rest = [d for d in range(64) if d not in (5, 9)]
    assert torch.equal(out[:n][:, :, rest], want[:n][:, :, rest])


def test_stream_lowest_and_huge_scores(pa):
    """Scores of thousands, of either sign: the running maximum keeps the weights in range."""
    for fmt in ("bf16", "nvfp4"):
        t = Rows(82, [(200, 9), (65, 17), (3, 3), (700, 300)], 8, 2, 128, 16, fmt, big_q=300.0)
        out, lse, _ = t.call(pa)
        t.compare(out, lse)


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_stream_scales(pa, scale):
    t = Rows(83, [(200, 9), (65, 17), (700, 300)], 8, 2, 128, 16, "bf16", 90, 5)
    t.scale = scale
    t.check(pa)
    u = Rows(84, [(200, 9), (65, 17), (700, 300)], 8, 2, 64, 16, "fp8", 90, 5)
    u.scale = scale
    u.check(pa)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("hq,hkv,D,window,first", [(8, 2, 128, 90, 5), (2, 2, 64, 0, 0), (4, 1, 256, 30, 0)])
@pytest.mark.parametrize("k_scale,sign", [(0.02, 1), (1e-7, 1), (1e-7, -1), (1e-20, 1)])
def test_stream_zero_and_tiny_queries(pa, fmt, hq, hkv, D, window, first, k_scale, sign):
    """Padding's zero queries, and ones at the end of bf16's range, attend to all that they see alike, however small the keys' scale."""
    t = Rows(85, [(200, 9), (65, 17), (700, 300), (40, 1)], hq, hkv, D, 16, fmt, window, first)
    t.q[::2, 0] = 0.0
    t.q[1::3, 1] *= 2.0 ** -126
    t.q[5] = 0.0
    t.scale *= sign
    if fmt == "bf16":
        t.scale *= k_scale
    else:
        t.scales = (k_scale, 0.02)
    t.check(pa)


def test_stream_is_decode_verify_and_tree(pa):
    """Within both sides' rounding: half a bf16 step of each output and of each weight."""
    rows = [(100, 5), (685, 5), (33, 5)]
    t = Rows(90, rows, 16, 4, 128, 32, extra=0)
    out, lse, _ = t.call(pa)
    q = t.q.view(3, 5, 16, 128)
    vo, vl = torch.empty_like(q), torch.empty(3, 5, 16, device="cuda")
    bt, lens = i32(t.table), i32([L for L, _ in rows])
    ref = t.reference()
    tol = 2 * (2.0 ** -8 * np.abs(ref[0]) + (2.0 ** -8 + 1e-4) * 1.01 * ref[2])
    pa.pa_verify_gqa(q, t.k, t.v, bt, lens, vo, vl, scale=t.scale, workspace=pa.workspace_for_gqa(q, t.k, bt))
    assert np.all(np.abs(f64(out) - f64(vo.view_as(out))) <= tol)
    assert np.all(np.abs(f64(lse) - f64(vl.view_as(lse))) <= 1e-4)
    mask = dev(np.array([2 ** (i + 1) - 1 for _ in rows for i in range(5)], np.int64))
    to, tl = torch.empty_like(t.q), torch.empty(15, 16, device="cuda")
    pa.pa_tree_gqa(*t.args(), mask, to, tl, max_query=5, scale=t.scale, workspace=pa.workspace_for_tree(t.q, t.k, bt, 5))
    assert np.all(np.abs(f64(out) - f64(to)) <= tol) and np.all(np.abs(f64(lse) - f64(tl)) <= 1e-4)


def test_stream_bitwise_repeatable_and_independent_of_page_order(pa):
    rows = [(1000, 12), (64, 64), (7, 2), (3000, 300)]
    for fmt in ("bf16", "fp8"):
        a, b = Rows(91, rows, 16, 2, 128, 16, fmt, 500, 20), Rows(91, rows, 16, 2, 128, 16, fmt, 500, 20, shuffle=False)
        (oa, la, _), (ob, lb, _), (oc, lc, _) = a.call(pa), b.call(pa), a.call(pa)
        assert torch.equal(oa, ob) and torch.equal(la, lb) and torch.equal(oa, oc) and torch.equal(la, lc)


def test_stream_captured_and_replayed_with_other_lengths(pa):
    """A graph of the call replays with new lengths and tables in the same arrays; a second graph shares the workspace."""
    first, second = Rows(92, [(300, 8), (90, 300 - 8)][:1] + [(400, 292)], 8, 2, 128, 16), Rows(93, [(400, 292), (250, 8)], 8, 2, 128, 16)
    args = [x.clone() for x in first.args()]
    args[3] = torch.zeros(2, 30, dtype=torch.int32, device="cuda")
    args[1], args[2] = (torch.zeros(60, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def load(t):
        a = t.args()
        for i in (0, 4, 5):
            args[i].copy_(a[i])
        args[3][:, :a[3].shape[1]].copy_(a[3])
        for i in (1, 2):
            args[i][:a[i].shape[0]].copy_(a[i])

    load(first)
    outs = [(torch.zeros_like(first.q), torch.zeros(first.q.shape[:2], device="cuda")) for _ in range(2)]
    ws = pa.workspace_for_stream(first.q, args[1], args[3], 300)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first.call(pa, 300, args=args, out=outs[0][0], lse=outs[0][1], ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for o, l in outs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            first.call(pa, 300, args=args, out=o, lse=l, ws=ws)
    for t in (second, first):
        load(t)
        for graph, (o, l) in zip(graphs, outs):
            graph.replay()
            torch.cuda.synchronize()
            t.compare(o, l)


def test_stream_two_streams(pa):
    """Two calls at once, each with its own workspace."""
    a, b = Rows(94, [(4000, 300)], 16, 2, 128, 16), Rows(95, [(3000, 7), (500, 90)], 16, 2, 128, 16, "fp8", 400, 9)
    xa, xb = a.args(), b.args()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    pre = [[torch.full(t.q.shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(t.q.shape[:2], 7.0, device="cuda")] for t in (a, b)]
    wa, wb = pa.workspace_for_stream(a.q, a.k, xa[3], 300), pa.workspace_for_stream(b.q, b.k, xb[3], 90)
    torch.cuda.synchronize()
    for _ in range(5):
        a.call(pa, args=xa, out=pre[0][0], lse=pre[0][1], ws=wa, stream=sa)
        b.call(pa, args=xb, out=pre[1][0], lse=pre[1][1], ws=wb, stream=sb.cuda_stream)
    torch.cuda.synchronize()
    a.compare(*pre[0])
    b.compare(*pre[1])


def test_stream_without_lse_and_granted(pa):
    t = Rows(96, [(300, 20), (90, 9), (500, 140)], 8, 2, 128, 16, "bf16", 100, 4)
    want, want_l = t.check(pa, num_splits=1)  # (one share: where rows are cut depends on all of them)
    out = torch.full(t.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    t.call(pa, out=out, num_splits=1)
    assert torch.equal(out, want)
    args = list(t.args())
    args[4] = i32([300, -5, 500])  # what a refused row's lengths say is not looked at
    out, lse, ws = t.call(pa, args=args, granted=i32([1, 0, 7]), num_splits=1)
    torch.cuda.synchronize()
    assert pa.pa_read_device_status(ws) == 0
    assert torch.equal(out[:20], want[:20]) and torch.equal(out[29:], want[29:]) and bool((out[20:29] == 7.0).all())
    assert torch.equal(lse[:20], want_l[:20]) and torch.equal(lse[29:], want_l[29:]) and bool((lse[20:29] == 7.0).all())


def test_stream_refuses_lengths_on_the_device(pa):
    """Bad rows set the status bit; the others are as without them."""
    good = Rows(97, [(300, 20), (200, 1)], 8, 2, 128, 16)
    want, want_l = good.check(pa)
    q, k, v, table, lens, start = good.args()
    for change in (dict(lens=[300, -1]), dict(lens=[300, 0]), dict(lens=[300, 100000]), dict(start=[0, 20, 19]),
                   dict(start=[0, 20, 50]), dict(start=[0, 20, 20 + 400])):
        ln, st = i32(change.get("lens", [300, 200])), i32(change.get("start", [0, 20, 21]))
        out, lse, ws = good.call(pa, max_query=25, args=(q, k, v, table, ln, st))
        torch.cuda.synchronize()
        assert pa.pa_read_device_status(ws) == pa.PA_DEV_BAD_LEN, change
        assert np.abs(f64(out[:20]) - f64(want[:20])).max() <= 0.05


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("splits", [0, 1, 40])
def test_stream_rows_beside_refused_lengths(pa, fmt, splits):
    """Rows before and behind a row with bad lengths are those of the 64-bit reference, and tokens behind the last row stay."""
    good = Rows(97, [(3000, 20), (200, 3), (900, 150)], 8, 2, 128, 16, fmt, 700, 9)
    o, l, spread, size = good.reference()
    q, k, v, table, _, _ = good.args()
    for lens, start in (([3000, -1, 900], [0, 20, 23, 173]), ([3000, 2, 900], [0, 20, 23, 173]), ([3000, 1 << 30, 900], [0, 20, 23, 173]),
                        ([3000, 200, 900], [0, 20, 200, 173]), ([3000, 200, 900], [0, 20, -5, 173])):
        out, lse, ws = good.call(pa, max_query=150, num_splits=splits, args=(q, k, v, table, i32(lens), i32(start)))
        torch.cuda.synchronize()
        assert pa.pa_read_device_status(ws) == pa.PA_DEV_BAD_LEN, (lens, start)
        assert bool((out[173:] == 7.0).all()) and bool((lse[173:] == 7.0).all())
        for s in (slice(0, 20), slice(23, 173))[:2 if start[2] == 23 else 1]:  # (a bad start makes the row behind it another one)
            R.check_tree(f64(out[s]), f64(lse[s]), o[s], l[s], spread[s], size[s], good.D, good.lost())


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_stream_bad_pages(pa, fmt):
    """A visited entry outside the pool sets the status bit and is not loaded; rows that do not visit it keep their bits."""
    t = Rows(98, [(300, 20), (500, 140), (40, 1)], 8, 2, 128, 16, fmt)
    want, want_l = t.check(pa, num_splits=1)
    for bad in (-1, 1 << 30, t.k.shape[0]):
        u = t.table.copy()
        u[1, 9] = bad
        args = list(t.args())
        args[3] = i32(u)
        out, lse, ws = t.call(pa, num_splits=1, args=args)
        torch.cuda.synchronize()
        assert pa.pa_read_device_status(ws) == pa.PA_DEV_BAD_PAGE
        assert torch.equal(out[:20], want[:20]) and torch.equal(out[160:161], want[160:161])


def test_stream_offsets_past_32_bits(pa):
    """Pages whose bytes, and whose values, lie behind 2^32 of the pool's."""
    for fmt, pages in (("bf16", 66000), ("fp8", 132000)):
        t = Rows(99, [(300, 20), (500, 140)], 16, 8, 128, 64, fmt, 200, 5, offset=pages)
        assert t.k.numel() > 1 << 32
        t.check(pa)
        del t
        torch.cuda.empty_cache()


# ------------------------------------------------------------------------------------------ pages released

def released(pa, c, in_place, ended, status=True):
    """Calls with the case's arrays; returns what the reference calls the same."""
    B = len(c["lens"])
    t = dict(lens=i32(c["lens"]), held=i32(c["held"]), start=i32(c["start"]), free=i32(c["free_list"]), count=i32([c["count"]]),
             table=i32(c["table"]))
    word = torch.zeros(1, dtype=torch.int32, device="cuda") if status else None
    outs = {} if in_place else dict(context_lens_out=i32([5] * B), held_pages_out=i32([5] * B), window_start_out=i32([5] * B),
                                    free_count_out=i32([5]), block_table_out=t["table"].clone())
    pa.pa_release_pages(t["lens"], t["held"], t["start"], t["free"], t["count"], t["table"], page_size=c["P"], window=c["window"],
                        first=c["first"], ended=None if ended is None else i32(ended), status=word, **outs)
    torch.cuda.synchronize()
    if not in_place:
        for name in ("lens", "held", "start"):
            assert t[name].tolist() == list(c[name]), "inputs stay"
        assert t["count"].tolist() == [c["count"]] and np.array_equal(t["table"].cpu().numpy(), c["table"])
    pick = lambda name, key: (outs[name] if outs else t[key]).cpu().numpy()  # noqa: E731
    return dict(table=pick("block_table_out", "table"), free_list=t["free"].cpu().numpy(), count=int(pick("free_count_out", "count")[0]),
                lens=pick("context_lens_out", "lens").tolist(), held=pick("held_pages_out", "held").tolist(),
                start=pick("window_start_out", "start").tolist(), bits=int(word[0]) if status else None)


def release_case(seed, B, P, most, window, first):
    rng = np.random.default_rng(seed)
    F = -(-first // P)
    lens = rng.integers(0, most + 1, B)
    held = np.minimum(-(-lens // P) + rng.integers(0, 2, B), -(-most // P) + 1)
    W = -(-most // P) + 2
    before = np.maximum(0, lens - rng.integers(0, 4 * P, B) + 1 - window) // P
    start = np.where(before > F, np.minimum(before, held), 0)
    total = int(held.sum()) + 3
    pages = rng.permutation(total)
    table, at = np.full((B, W), -1, np.int64), 0
    for b in range(B):
        for j in range(held[b]):
            if F <= j < start[b]:
                continue
            table[b, j] = pages[at]
            at += 1
    free = total - at
    count = int(rng.integers(0, free + 1))
    free_list = np.full(total, -9, np.int64)
    free_list[:count] = pages[at:at + count]
    return dict(lens=lens.tolist(), held=held.tolist(), start=start.tolist(), free_list=free_list, count=count, table=table, P=P,
                window=window, first=first)


def same(got, want):
    assert np.array_equal(got["table"], want["table"]) and np.array_equal(got["free_list"], want["free_list"])
    for k in ("count", "lens", "held", "start"):
        assert got[k] == want[k], k
    if got["bits"] is not None:
        assert got["bits"] == want["bits"]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,P,most,window,first", [(1, 16, 100, 10, 4), (7, 8, 500, 64, 0), (33, 1, 90, 1, 3), (64, 16, 3000, 100, 33),
                                                   (600, 32, 900, 1, 32), (1025, 7, 200, 9, 1000), (8192, 16, 64, 20, 1),
                                                   (5, 16, 40000, 2 ** 31 - 1, 0), (300, 16, 9000, 256, 2 ** 31 - 1), (40, 16, 30000, 7, 5)])
def test_release(pa, in_place, B, P, most, window, first):
    for seed in (1, 2):
        c = release_case(seed + B, B, P, most, window, first)
        ended = (np.random.default_rng(seed).integers(0, 5, B) == 0).astype(int).tolist()
        for e in (None, ended, [1] * B):
            args = (c["lens"], c["held"], c["start"], c["free_list"], c["count"], c["table"], P, len(c["free_list"]), window, first, e)
            same(released(pa, c, in_place, e), S.release(*args))


def test_release_twice_gives_nothing_more(pa):
    c = release_case(5, 40, 16, 4000, 300, 20)
    once = released(pa, c, True, None)
    c.update(lens=once["lens"], held=once["held"], start=once["start"], free_list=once["free_list"], count=once["count"], table=once["table"])
    twice = released(pa, c, True, None)
    same(twice, {**once, "bits": 0})


def test_release_of_bad_states(pa):
    c = release_case(6, 12, 16, 3000, 100, 33)
    W = c["table"].shape[1]
    c["lens"][1], c["held"][2], c["held"][3], c["start"][4] = -3, -1, W + 1, -1
    c["start"][5] = c["held"][5] + 1
    c["lens"][6] = 2 ** 31 - 1  # longer than what it holds: all its pages but the first ones'
    c["table"][7, :c["held"][7]] = 1 << 20
    c["lens"][7] = c["held"][7] * 16
    for ended in (None, [0, 1] * 6):
        args = (c["lens"], c["held"], c["start"], c["free_list"], c["count"], c["table"], 16, len(c["free_list"]), 100, 33, ended)
        for in_place in (False, True):
            got = released(pa, c, in_place, ended)
            same(got, S.release(*args))
            assert got["bits"] & pa.PA_DEV_BAD_LEN
    # a list without room, a count out of range
    c = release_case(7, 30, 16, 3000, 100, 33)
    for n, count in ((10, 4), (10, 10), (10, 11), (10, -1)):
        d = dict(c, free_list=c["free_list"][:n], count=count)
        args = (d["lens"], d["held"], d["start"], d["free_list"], count, d["table"], 16, n, 100, 33, None)
        same(released(pa, d, True, None), S.release(*args))


def test_release_without_status_or_rows(pa):
    c = release_case(8, 3, 16, 900, 100, 3)
    same(released(pa, c, False, None, status=False), S.release(c["lens"], c["held"], c["start"], c["free_list"], c["count"], c["table"], 16,
                                                              len(c["free_list"]), 100, 3))
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    for out in (None, z(1)):
        pa.pa_release_pages(z(0), z(0), z(0), z(5), i32([3]), z(0, 4), page_size=8, window=4, free_count_out=out)
        assert out is None or out.tolist() == [3]


@pytest.mark.parametrize("in_place", [False, True])
def test_plan_says_that_an_ended_row_gives_no_pages(pa, in_place):
    """A row whose window has passed pages and that ends in the plan instead of the release: what goes onto the list is what the table
    holds, and the status says that some of it are no pages, in that call already."""
    P, pages, W = 16, 40, 12
    for first, bits in ((20, pa.PA_DEV_BAD_PAGE), (200, 0)):
        lens, held, start = i32([150, 40]), i32([10, 3]), i32([0, 0])
        table = i32(np.arange(2 * W).reshape(2, W))
        free, count, st = i32([30, 31, 32] + [-9] * (pages - 3)), i32([3]), i32([0])
        pa.pa_release_pages(lens, held, start, free, count, table, page_size=P, window=64, first=first, status=st)
        gone = 3 if first == 20 else 0  # pages 2 to 4 lie between the first tokens' two and the window
        assert int(count) == 3 + gone and int(st) == 0
        row, before = table[0, :10].tolist(), int(count)
        out = {} if in_place else {"context_lens_out": i32([0] * 2), "held_pages_out": i32([0] * 2), "free_count_out": i32([0])}
        pa.pa_plan_step(lens, i32([-1, 0]), held, free, count, table, i32([0] * 3), dev([0] * 4, torch.int64), i32([0] * 4),
                        page_size=P, status=st, **out)
        after = int(out.get("free_count_out", count))
        assert int(st) == bits and after == before + 10 and free[before:after].tolist() == row
        assert row.count(-1) == gone


# ------------------------------------------------------------------------------------------ steps together

@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("captured", [False, True])
def test_streams_of_steps_in_bounded_memory(pa, fmt, captured):
    """Plan, rotation + write, attention and release, step after step, in a pool that could not hold the streams whole; chunks, then single
    tokens, a row that ends and one that begins in its place.  Each step's attention against the whole history."""
    B, hq, hkv, D, P, window, first, pages = 3, 8, 2, 128, 16, 64, 5, 40
    rng = np.random.default_rng(5)
    scales = {"bf16": (1.0, 1.0), "fp8": (0.02, 0.02), "nvfp4": (0.25, 0.25)}[fmt]
    more = {} if fmt == "bf16" else {"k_scale": scales[0], "v_scale": scales[1]}
    sfx = "" if fmt == "bf16" else "_" + fmt
    width = D if fmt == "bf16" else R.row_bytes(fmt, D)
    z = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    kind = torch.bfloat16 if fmt == "bf16" else torch.uint8
    k_pool, v_pool = z(pages, P, hkv, width, d=kind), z(pages, P, hkv, width, d=kind)
    lens, held, start = z(B), z(B), z(B)
    free, count = i32(rng.permutation(pages)), i32([pages])
    W, T = 64, 160
    table, qs, slots, pos, granted, status, ended = z(B, W), z(B + 1), z(T, d=torch.int64), z(T), z(B), z(1), z(B)
    news = z(B)
    x = torch.zeros(T, hq + 2 * hkv, D, dtype=torch.bfloat16, device="cuda")
    q, out, lse = z(T, hq, D, d=torch.bfloat16), z(T, hq, D, d=torch.bfloat16), z(T, hq, d=torch.float32)
    angle = torch.rand(W * P, D // 2, generator=torch.Generator().manual_seed(1)) * 6.28
    cs = torch.cat((angle.cos(), angle.sin()), -1).cuda()
    ws = pa.workspace_for_stream(q, k_pool, table, T)

    def step():
        pa.pa_plan_step(lens, news, held, free, count, table, qs, slots, pos, page_size=P, granted=granted, status=status)
        getattr(pa, "pa_qk_norm_rope_write" + sfx)(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], None, None, cs, pos, slots, q,
                                                   k_pool, v_pool, status=status, **more)
        getattr(pa, "pa_stream_gqa" + sfx)(q, k_pool, v_pool, table, lens, qs, out, lse, max_query=T, scale=D ** -0.5, window=window,
                                           first=first, workspace=ws, granted=granted, **more)
        pa.pa_release_pages(lens, held, start, free, count, table, page_size=P, window=window, first=first, ended=ended, status=status)

    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()  # (of no tokens)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    hist = [([], []) for _ in range(B)]  # each row's keys and values as the cache holds them
    length = [0] * B
    peak = 0
    chunks = [[100, 33, 7], [50, 100, 1], [1, 120, 1], [90, 0, 60]] + [[1, 1, 1]] * 40 + [[1, 1, 0]] + [[1, 1, 30]] + [[1, 70, 1]] * 4
    for i, new in enumerate(chunks):
        end = [0, 0, 1 if i == 44 else 0]  # row 2 ends with that step and begins anew in the next
        news.copy_(i32(new))
        ended.copy_(i32(end))
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16))
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert int(status) == 0 and pa.pa_read_device_status(ws) == 0 and granted.tolist() == [1] * B
        kk = R.pool_values(raw(k_pool), fmt, D, scales[0]).reshape(pages * P, hkv, D)
        vv = R.pool_values(raw(v_pool), fmt, D, scales[1]).reshape(pages * P, hkv, D)
        sl, at, parts = slots.tolist(), 0, []
        for b, n in enumerate(new):
            for j in range(n):
                hist[b][0].append(kk[sl[at + j]])
                hist[b][1].append(vv[sl[at + j]])
            length[b] += n
            if n:
                parts.append(S.stream_attention(f64(q[at:at + n]), np.array(hist[b][0]), np.array(hist[b][1]), length[b], D ** -0.5, window, first))
            at += n
        ref = [np.concatenate(y) for y in zip(*parts)]
        lost = 0.0 if fmt == "bf16" else 2.0 ** -32 * max(length) * float(np.abs(vv).max())
        R.check_tree(f64(out[:at]), f64(lse[:at]), *ref, D, lost)
        for b in range(B):
            if end[b]:
                hist[b], length[b] = ([], []), 0
        assert lens.tolist() == length
        used = pages - int(count)
        for b in range(B):
            used_b = -(-length[b] // P) - max(0, max(0, length[b] + 1 - window) // P - 1)
            used -= used_b
        assert used == 0, "the rows hold the first tokens' pages and the window's"
        peak = max(peak, sum(length))
    assert peak > pages * P, "more tokens than the pool holds"
    everything = sorted(free.tolist()[:int(count)] + [int(e) for b in range(B) for e in table[b, :int(held[b])].tolist() if e >= 0])
    assert everything == list(range(pages)), "each page is somebody's, once"
