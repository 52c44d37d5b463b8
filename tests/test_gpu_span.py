"""GPU parity of the span operators (chunks over a paged cache, sliding windows with sinks, e4m3 caches)
against the float64 oracle, through the C ABI.

Tolerances.  An output is sum_u w_u v_u with weights w_u >= 0 of sum 1; ``size`` is the same sum over |v|.
bf16: every weight is rounded to bf16 once (relative 2^-8) and the result once (2^-8 of at most ``size``), so
|error| <= 2^-7 size, plus the fp32 part below, which 2^-12 size covers here.  fp32: a score is a sum of d
products, off by at most (d + 2) 2^-24 S with S = scale sum_e |q_e k_e|; with the factor log2 e, the subtraction
and the exponential each off by a few last places of |z| <= S, a weight is off by a relative (d + 8) 2^-24 S
+ 2^-21, both in the sum of the weights and in the sum over v, and the sums themselves by (n + 4) 2^-24 for n
positions: |error| <= (2 (d + 8) S + 2 n + 32) 2^-24 size.
"""
import numpy as np
import pytest
import torch

import packed_question_isolated_gb300 as kev
import workloads as W
from oracle import kev_oracle as O

pytestmark = pytest.mark.gpu

PAGE = 128
TD = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


class Span:
    """Device buffers of one batch: packed rows, a paged cache with scattered blocks, and its twin on the host."""

    def __init__(self, seed, lens, prefix, h_q, h_kv, d, dtype="bf16", pool="bf16", gaps=0, spare=2, fill=None, width=None,
                 order=None):
        g = np.random.default_rng(seed)
        n = len(lens)
        self.lens, self.prefix, self.h_q, self.h_kv, self.d = list(lens), list(prefix), h_q, h_kv, d
        self.dtype, self.pool = dtype, pool
        at, self.intervals = 0, np.zeros((n, 2), np.int32)
        for i in (order if order is not None else range(n)):
            at += gaps
            self.intervals[i] = (at, at + lens[i])
            at += lens[i]
        self.T = at + gaps
        self.q, self.k, self.v = (torch.from_numpy(g.standard_normal((self.T, h, d), dtype=np.float32)).to(TD[dtype]).cuda()
                                  for h in (h_q, h_kv, h_kv))
        pages = [-(-(p + m) // PAGE) for p, m in zip(prefix, lens)]
        self.n_blocks, self.width = sum(pages) + spare, width or max(max(pages), 1)
        ids, at = g.permutation(self.n_blocks), 0
        self.table = np.full((n, self.width), -1, np.int32)
        for i, m in enumerate(pages):
            self.table[i, :m] = ids[at:at + m]
            at += m
        shape = (self.n_blocks, h_kv, PAGE, d)
        self.pools = []
        for _ in range(2):
            x = torch.from_numpy(g.standard_normal(shape, dtype=np.float32))
            if fill is not None:
                x.fill_(fill)
            if pool == "e4m3":
                code, s = O.quantise_rows(x.numpy())
                self.pools.append((torch.from_numpy(code).float().to(TD["e4m3"]).cuda(), torch.from_numpy(s).cuda()))
            else:
                self.pools.append((x.to(TD[pool]).cuda(), None))
        self.shape = kev.make_shape(h_q, h_kv, d, dtype)
        self.bytes = kev.kev_paged_workspace_size(n, self.T, self.shape)
        self.ws = torch.full((self.bytes,), 0xff, dtype=torch.uint8, device="cuda")
        self.status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        self.out = torch.full((self.T, h_q, d), float("nan"), dtype=TD[dtype], device="cuda")
        self.to_device()

    def to_device(self):
        self.iv = torch.from_numpy(self.intervals).cuda()
        self.pre = torch.from_numpy(np.asarray(self.prefix, np.int32)).cuda()
        self.tab = torch.from_numpy(self.table).cuda()
        (k, ks), (v, vs) = self.pools
        self.cache = kev.make_paged_cache(k, v, self.tab, self.width, self.n_blocks, self.pool, ks, vs)

    def end(self):
        return self.shape, self.ws, self.bytes, self.status

    def write(self, **kw):
        return kev.kev_paged_write(self.k, self.v, self.T, self.iv, len(self.lens), self.pre, self.cache, *self.end(), **kw)

    def chunk(self, window=0, sinks=0, max_chunk=0, write=True, **kw):
        return kev.kev_chunk_attn_paged(self.q, self.k if write else None, self.v if write else None, self.T, self.iv,
                                        len(self.lens), self.pre, max_chunk, self.cache, window, sinks, self.out, *self.end(),
                                        **kw)

    def packed(self, window, sinks, **kw):
        return kev.kev_prefill_attn_window(self.q, self.k, self.v, self.T, self.iv, len(self.lens), window, sinks, self.out,
                                           *self.end(), **kw)

    def ok(self):
        assert kev.kev_read_status(self.status) == 0

    def stored(self):
        """What the cache holds, as float64 [n_blocks, h_kv, PAGE, d] for K and V."""
        return [(p.float().cpu().numpy().astype(np.float64) if s is None else
                 p.float().cpu().numpy().astype(np.float64) * s.cpu().numpy().astype(np.float64)[..., None])
                for p, s in self.pools]

    def caches(self):
        """Question by question, positions 0 .. P + L - 1 of the cache: [(K, V)] of [P + L, h_kv, d]."""
        pk, pv = self.stored()
        res = []
        for i, (m, p) in enumerate(zip(self.lens, self.prefix)):
            b = np.maximum(self.table[i, :-(-(p + m) // PAGE)], 0)
            res.append(tuple(x[b].transpose(0, 2, 1, 3).reshape(-1, self.h_kv, self.d)[:p + m] for x in (pk, pv)))
        return res

    def check(self, keys, values, window, sinks, prefix=None):
        q = self.q.float().cpu().numpy().astype(np.float64)
        pre = self.prefix if prefix is None else prefix
        ref, size = O.span_attention(q, keys, values, pre, self.intervals, window, sinks)
        got = self.out.float().cpu().numpy().astype(np.float64)
        assert np.isfinite(got).all()
        if self.dtype == "bf16":
            tol = (2.0 ** -7 + 2.0 ** -12) * size
        else:
            n = max([p + m for p, m in zip(pre, self.lens)])
            with np.errstate(invalid="ignore"):
                top = max([np.nanmax(np.abs(np.where(np.isfinite(k), k, 0))) for k in keys if k.size] + [0])
            s = np.abs(q).sum(-1, keepdims=True) * top / np.sqrt(self.d)
            tol = (2 * (self.d + 8) * s + 2 * n + 32) * 2.0 ** -24 * size
        bad = np.abs(got - ref) > tol + 1e-30
        assert not bad.any(), (int(bad.sum()), float(np.abs(got - ref).max()), np.argwhere(bad)[:4].tolist())
        inside = np.zeros(self.T, bool)
        for b, e in self.intervals:
            inside[b:e] = True
        assert (got[~inside] == 0).all()


def _kv(x):
    return [a for a, _ in x], [b for _, b in x]


# lens, prefix, h_q, h_kv, d
SHAPES = [
    ([1, 1, 1, 1], [0, 127, 128, 700], 8, 2, 128),
    ([3, 0, 130, 1, 257], [5, 9, 250, 1000, 0], 28, 4, 128),
    ([70, 33], [1, 383], 4, 4, 64),
    ([200, 1], [64, 2000], 16, 1, 128),
    ([2, 5, 1], [126, 0, 900], 12, 4, 64),
]
MASKS = [(0, 0), (1, 0), (100, 4), (128, 130), (300, 1)]


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("dtype,pool", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32"), ("fp32", "e4m3")])
def test_chunk_against_oracle(dtype, pool, shape, mask):
    lens, prefix, h_q, h_kv, d = SHAPES[shape]
    b = Span(100 + shape, lens, prefix, h_q, h_kv, d, dtype, pool, gaps=shape % 2)
    b.chunk(*mask)
    b.ok()
    b.check(*_kv(b.caches()), *mask)


@pytest.mark.parametrize("dtype,pool", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "e4m3")])
@pytest.mark.parametrize("h_q,h_kv,d", [(8, 2, 128), (28, 4, 128), (16, 1, 128), (6, 6, 64), (8, 2, 64)])
@pytest.mark.parametrize("mask", [(0, 0), (200, 4)])
def test_decode_steps_with_max_chunk(dtype, pool, h_q, h_kv, d, mask):
    """One token per question, told so: caches from empty to long, a dropped question, unsorted intervals."""
    b = Span(7 + h_q + d, [1, 1, 0, 1, 1, 1], [0, 128, 50, 511, 2500, 640], h_q, h_kv, d, dtype, pool, order=[3, 0, 1, 5, 4, 2])
    b.chunk(*mask, max_chunk=1)
    b.ok()
    b.check(*_kv(b.caches()), *mask)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("h_q,h_kv,d,mask", [(8, 2, 128, (0, 0)), (28, 4, 128, (150, 3)), (16, 1, 64, (0, 0)), (4, 4, 64, (64, 1))])
def test_mixed_rounds_of_chunks_and_single_tokens(pool, h_q, h_kv, d, mask):
    """A scheduler's round: many questions with one or two tokens beside a few longer chunks and an empty one."""
    r = np.random.default_rng(h_q)
    lens = [1] * 30 + [150, 2, 0, 40, 3]
    prefix = r.integers(0, 700, len(lens)).tolist()
    b = Span(70 + h_q, lens, prefix, h_q, h_kv, d, "bf16", pool, gaps=1, order=r.permutation(len(lens)).tolist())
    b.chunk(*mask)
    b.ok()
    b.check(*_kv(b.caches()), *mask)


@pytest.mark.parametrize("n,prefix", [(1, 30000), (2, 9000), (300, 40)])
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_one_long_cache_is_split_and_many_short_ones_are_not(n, prefix, pool):
    r = np.random.default_rng(n)
    b = Span(40 + n, [1] * n, r.integers(prefix // 2, prefix + 1, n).tolist(), 8, 2, 128, "bf16", pool)
    b.chunk(max_chunk=1)
    b.ok()
    b.check(*_kv(b.caches()), 0, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("h_q,h_kv,d", [(8, 2, 128), (7, 1, 64), (3, 3, 128), (28, 4, 64)])
@pytest.mark.parametrize("mask", [(1, 0), (17, 3), (128, 0), (200, 129), (5000, 2), (0, 0)])
def test_packed_window_against_oracle(dtype, h_q, h_kv, d, mask):
    lens = [1, 150, 0, 77, 300, 129]
    b = Span(60 + h_q, lens, [0] * 6, h_q, h_kv, d, dtype, gaps=2, order=[4, 1, 0, 5, 3, 2])
    b.packed(*mask)
    b.ok()
    k, v = (x.float().cpu().numpy().astype(np.float64) for x in (b.k, b.v))
    b.check([k[s:e] for s, e in b.intervals], [v[s:e] for s, e in b.intervals], *mask)


@pytest.mark.parametrize("dtype,d,pool", [("bf16", 128, "e4m3"), ("bf16", 64, "e4m3"), ("fp32", 128, "e4m3"), ("fp32", 64, "e4m3"),
                                          ("bf16", 128, "bf16"), ("bf16", 64, "bf16"), ("fp32", 64, "fp32"),
                                          ("fp32", 128, "fp32")])
@pytest.mark.parametrize("h_kv", [1, 3, 8, 17])
def test_write_and_read_back(dtype, d, pool, h_kv):
    """The cache after a write equals the oracle's rows bit for bit, nothing else is touched, and reading gives
    code * scale rounded once."""
    b = Span(80 + h_kv, [1, 200, 0, 129, 5], [3, 127, 9, 0, 250], h_kv, h_kv, d, dtype, pool, gaps=1)
    if pool == "e4m3":  # rows of zeros, tiny and huge rows
        b.k[3] = 0
        b.k[5] *= 1e-30
        b.v[7] *= 1e30
    raw = torch.uint8 if pool == "e4m3" else torch.int16 if pool == "bf16" else torch.int32
    want = [(p.view(raw).clone(), None if s is None else s.clone()) for p, s in b.pools]
    for x, (p, s) in zip((b.k, b.v), want):
        for i, (m, pre) in enumerate(zip(b.lens, b.prefix)):
            for j in range(m):
                row = x[b.intervals[i, 0] + j]
                blk, r = int(b.table[i, (pre + j) // PAGE]), (pre + j) % PAGE
                if pool == "e4m3":
                    code, sc = O.quantise_rows(row.float().cpu().numpy())
                    p[blk, :, r] = torch.from_numpy(code).float().to(TD["e4m3"]).view(raw).cuda()
                    s[blk, :, r] = torch.from_numpy(sc).cuda()
                else:
                    p[blk, :, r] = row.view(raw)
    b.write()
    b.ok()
    for (p, s), (wp, ws) in zip(b.pools, want):
        assert torch.equal(p.view(raw), wp)
        assert s is None or torch.equal(s, ws)
    ko, vo = torch.full_like(b.k, -7.0), torch.full_like(b.v, -9.0)
    kev.kev_paged_read(ko, vo, b.T, b.iv, len(b.lens), b.pre, b.cache, *b.end())
    b.ok()
    for got, mark, (p, s) in ((ko, -7.0, b.pools[0]), (vo, -9.0, b.pools[1])):
        wantrow = torch.full_like(got, mark)
        for i, (m, pre) in enumerate(zip(b.lens, b.prefix)):
            for j in range(m):
                blk, r = int(b.table[i, (pre + j) // PAGE]), (pre + j) % PAGE
                x = p[blk, :, r].float()
                wantrow[b.intervals[i, 0] + j] = (x if s is None else x * s[blk, :, r, None]).to(got.dtype)
        assert torch.equal(got, wantrow)


COPIES = [([1] * 32, [i * 9 for i in range(32)], 8), ([1], [128], 5), ([512], [77], 1), ([1, 0, 300, 129, 0, 60], [3, 5, 127, 0, 0, 250], 3),
          ([1] * 512, [i % 140 for i in range(512)], 1), ([0, 0], [4, 0], 2)]


@pytest.mark.parametrize("dtype,d,pool", [("bf16", 128, "e4m3"), ("fp32", 64, "e4m3"), ("bf16", 64, "bf16"), ("fp32", 128, "fp32")])
@pytest.mark.parametrize("lens,prefix,h_kv", COPIES)
def test_copies_of_small_calls_equal_those_of_large_ones(lens, prefix, h_kv, dtype, d, pool):
    """Up to 512 tokens take one kernel; the same batch with rows of no question behind it takes two."""
    order = np.random.default_rng(5).permutation(len(lens)).tolist()
    b = Span(90, lens, prefix, h_kv, h_kv, d, dtype, pool, order=order, spare=3)
    more = 600
    k, v = (torch.cat([x, torch.zeros((more, h_kv, d), dtype=TD[dtype], device="cuda")]) for x in (b.k, b.v))
    n, ws = len(lens), torch.full((kev.kev_paged_workspace_size(len(lens), b.T + more, b.shape),), 0xff, dtype=torch.uint8, device="cuda")
    start = [(p.view(torch.uint8).clone(), None if s is None else s.clone()) for p, s in b.pools]
    b.write()
    b.ok()
    small = [(p.view(torch.uint8).clone(), None if s is None else s.clone()) for p, s in b.pools]
    for (p, s), (p0, s0) in zip(b.pools, start):
        p.view(torch.uint8).copy_(p0)
        if s is not None:
            s.copy_(s0)
    end = (b.shape, ws, ws.numel(), b.status)
    kev.kev_paged_write(k, v, b.T + more, b.iv, n, b.pre, b.cache, *end)
    b.ok()
    for (p, s), (p0, s0), (p1, _) in zip(b.pools, small, start):
        assert torch.equal(p.view(torch.uint8), p0) and (s is None or torch.equal(s, s0))
        assert b.T == 0 or not torch.equal(p0, p1)
    got = []
    for t in (b.T, b.T + more):
        ko, vo = torch.full_like(k, -7.0), torch.full_like(v, -9.0)
        kev.kev_paged_read(ko, vo, t, b.iv, n, b.pre, b.cache, *end)
        b.ok()
        got.append((ko, vo))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("what", ["overlap", "nested", "outside", "reversed", "prefix", "overflow", "range", "negative", "twice", "two"])
@pytest.mark.parametrize("more", [0, 600])
def test_copies_check_before_they_write(what, more):
    b = Span(104, [5, 9, 1], [130, 40, 0], 4, 2, 128, "bf16", "e4m3")
    if what == "overlap":
        b.intervals[1, 0] -= 1
    elif what == "nested":
        b.intervals[2] = (2, 3)
    elif what == "outside":
        b.intervals[2, 1] = b.T + more + 1
    elif what == "reversed":
        b.intervals[0] = b.intervals[0][::-1]
    elif what == "prefix":
        b.prefix[1] = -1
    elif what == "overflow":
        b.prefix[1] = b.width * PAGE - 8
    elif what == "range":
        b.table[0, 1] = b.n_blocks
    elif what == "negative":
        b.table[1, 0] = -1
    elif what == "twice":
        b.table[1, 0] = b.table[0, 1]
    else:  # a block used twice and an overlap: the overlap is reported
        b.table[1, 0] = b.table[0, 1]
        b.intervals[2] = (2, 3)
    b.to_device()
    code = O.validate_span(b.intervals, b.T + more, b.prefix, b.table, b.n_blocks, attend=False)
    want = CODES[O.INTERVALS if what == "two" else code]
    k, v = (torch.cat([x, torch.ones((more, 2, 128), dtype=x.dtype, device="cuda")]) for x in (b.k, b.v))
    ws = torch.full((kev.kev_paged_workspace_size(3, b.T + more, b.shape),), 0xff, dtype=torch.uint8, device="cuda")
    before = [(p.view(torch.uint8).clone(), s.clone()) for p, s in b.pools] + [(k.clone(), v.clone())]
    for f in (kev.kev_paged_write, kev.kev_paged_read):
        b.status.fill_(-1)
        assert f(k, v, b.T + more, b.iv, 3, b.pre, b.cache, b.shape, ws, ws.numel(), b.status) == 0
        assert kev.kev_read_status(b.status) == want
    for (p, s), (p0, s0) in zip([(p.view(torch.uint8), s) for p, s in b.pools] + [(k, v)], before):
        assert torch.equal(p, p0) and torch.equal(s, s0)


def test_rows_with_nan_or_infinity_read_back_as_nan():
    b = Span(90, [4], [10], 2, 2, 128, "bf16", "e4m3")
    b.k[1, 0, 5], b.k[2, 1, 77] = float("nan"), float("inf")
    b.write()
    ko, vo = torch.empty_like(b.k), torch.empty_like(b.v)
    kev.kev_paged_read(ko, vo, b.T, b.iv, 1, b.pre, b.cache, *b.end())
    b.ok()
    nan = torch.isnan(ko.float()).all(-1).cpu()
    assert nan.tolist() == [[False, False], [True, False], [False, True], [False, False]]
    assert torch.isfinite(ko.float().cpu()[~nan]).all() and torch.isfinite(vo.float()).all()


@pytest.mark.parametrize("dtype,pool", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32")])
@pytest.mark.parametrize("lens,prefix,mask,max_chunk", [([1, 1, 1], [300, 129, 5], (100, 2), 1), ([1, 1], [300, 129], (0, 0), 1),
                                                        ([40, 1, 150], [300, 129, 5], (100, 2), 0), ([200, 3], [0, 260], (0, 0), 0)])
def test_masked_positions_may_hold_anything(dtype, pool, lens, prefix, mask, max_chunk):
    """NaN and infinities past the end of every cache, in blocks nobody uses and in positions out of the window
    do not reach the result."""
    b = Span(95, lens, prefix, 8, 2, 128, dtype, pool)
    b.write()
    keep = np.zeros((b.n_blocks, PAGE), bool)
    for i, (m, p) in enumerate(zip(lens, prefix)):
        for x in range(p, p + m):
            for u in np.flatnonzero(O.span_visible(x, x + 1, *mask)):
                keep[b.table[i, u // PAGE], u % PAGE] = True
    poison = torch.from_numpy(~keep).cuda()
    for z, (p, s) in enumerate(b.pools):
        bad = float("nan") if z else float("inf")
        if s is None:
            p[poison[:, None, :].expand(-1, b.h_kv, -1)] = bad
        else:
            p.view(torch.uint8)[poison[:, None, :].expand(-1, b.h_kv, -1)] = 0x7f
            s[poison[:, None, :].expand(-1, b.h_kv, -1)] = bad
    caches = b.caches()
    b.chunk(*mask, max_chunk=max_chunk, write=False)
    b.ok()
    b.check(*_kv(caches), *mask)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_packed_neighbours_and_later_tokens_may_hold_anything(dtype):
    """A question's rows do not see a neighbour's NaN, nor earlier tokens a later token's."""
    b = Span(97, [100, 60, 130], [0] * 3, 4, 2, 128, dtype)
    for x in (b.k, b.v):
        x[100:160] = float("nan")  # question 1
        x[160 + 70] = float("inf")  # question 2, position 70
    k, v = (x.float().cpu().numpy().astype(np.float64) for x in (b.k, b.v))
    b.packed(50, 2)
    b.ok()
    got = b.out.float().cpu().numpy()
    clean = list(range(100)) + [160 + j for j in range(130) if not 70 <= j < 120]
    ref, size = O.span_attention(b.q.float().cpu().numpy().astype(np.float64), [k[s:e] for s, e in b.intervals],
                                 [v[s:e] for s, e in b.intervals], [0] * 3, b.intervals, 50, 2)
    assert np.isfinite(got[clean]).all()
    assert (np.abs(got - ref)[clean] <= (2.0 ** -7 + 2.0 ** -12) * size[clean]).all()
    assert np.isnan(got[100:160]).all()


@pytest.mark.parametrize("scale", [30.0, 1000.0])
@pytest.mark.parametrize("dtype,pool", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32")])
def test_large_scores_and_growing_maximum(dtype, pool, scale):
    """Scores of hundreds whose maximum keeps moving along the cache: the running maximum has to follow."""
    for lens, prefix, mc in (([1, 1], [900, 130], 1), ([40, 130], [900, 130], 0)):
        b = Span(98, lens, prefix, 4, 2, 64, dtype, pool)
        b.q.mul_(scale)
        b.write()
        for i, (m, p) in enumerate(zip(lens, prefix)):  # keys grow along the cache
            for pg in range(-(-(p + m) // PAGE)):
                blk = int(b.table[i, pg])
                kp, ks = b.pools[0]
                if ks is None:
                    kp[blk] *= 0.2 * (pg + 1)
                else:
                    ks[blk] *= 0.2 * (pg + 1)
        b.chunk(max_chunk=mc, write=False)
        b.ok()
        q = b.q.float().cpu().numpy().astype(np.float64)
        ref, size = O.span_attention(q, *_kv(b.caches()), prefix, b.intervals)
        got = b.out.float().cpu().numpy()
        assert np.isfinite(got).all()
        # a score is off by (d + 8) 2^-24 S, S = scale sum |q k|: the weights by as much, relatively
        top = max(float(np.abs(k).max()) for k, _ in b.caches())
        s = np.abs(q).sum(-1, keepdims=True) * top / 8.0
        rel = 2 * 72 * s * 2.0 ** -24 + (2.0 ** -7 + 2.0 ** -12 if dtype == "bf16" else 2.0 ** -14)
        assert (np.abs(got - ref) <= np.minimum(rel, 2.0) * size + 1e-30).all()


def test_scores_of_minus_infinity_and_of_the_lowest_value():
    """A key whose score is -inf or the lowest finite one takes no part; the others are as without it."""
    b = Span(99, [1, 1], [200, 300], 2, 2, 128)
    b.q.abs_()
    b.write()
    kp = b.pools[0][0]
    kp[b.table[0, 0], :, 7] = -float("inf")
    kp[b.table[1, 1], :, 9] = torch.finfo(torch.bfloat16).min
    b.chunk(write=False, max_chunk=1)
    b.ok()
    b.check(*_kv(b.caches()), 0, 0)


def test_pages_out_of_the_window_need_no_block():
    b = Span(101, [1, 3], [1000, 700], 4, 2, 128, "bf16", "e4m3")
    for mask in ((200, 3), (130, 0)):
        table = b.table.copy()
        for i, (m, p) in enumerate(zip(b.lens, b.prefix)):
            first = max(0, p - mask[0] + 1) // PAGE
            table[i, (1 if mask[1] else 0):first] = -5
        b.tab.copy_(torch.from_numpy(table))
        b.chunk(*mask)
        b.ok()
        b.check(*_kv(b.caches()), *mask)


CODES = {O.INTERVALS: kev.binding.KEV_ERR_INTERVALS, O.PREFIX: kev.binding.KEV_ERR_PREFIX,
         O.SLOT_OVERFLOW: kev.binding.KEV_ERR_SLOT_OVERFLOW, O.SLOT: kev.binding.KEV_ERR_SLOT}
ERRORS = [
    ("overlap", O.INTERVALS), ("outside", O.INTERVALS), ("reversed", O.INTERVALS), ("max_chunk", O.INTERVALS),
    ("prefix", O.PREFIX), ("overflow", O.SLOT_OVERFLOW), ("range", O.SLOT), ("negative", O.SLOT), ("twice", O.SLOT),
]


@pytest.mark.parametrize("what,code", ERRORS)
def test_device_errors_write_nothing(what, code):
    b = Span(102, [5, 9], [130, 40], 4, 2, 128, "bf16", "e4m3")
    mc = 0
    if what == "overlap":
        b.intervals[1, 0] -= 1
    elif what == "outside":
        b.intervals[1, 1] += 1
    elif what == "reversed":
        b.intervals[0] = b.intervals[0][::-1]
    elif what == "max_chunk":
        mc = 8
    elif what == "prefix":
        b.prefix[1] = -1
    elif what == "overflow":
        b.prefix[1] = b.width * PAGE - 8
    elif what == "range":
        b.table[0, 1] = b.n_blocks
    elif what == "negative":
        b.table[0, 0] = -1
    else:
        b.table[1, 0] = b.table[0, 0]
    b.to_device()
    assert O.validate_span(b.intervals, b.T, b.prefix, b.table, b.n_blocks, mc) == code
    before = [(p.view(torch.uint8).clone(), s.clone()) for p, s in b.pools]
    assert b.chunk(max_chunk=mc) == 0
    assert kev.kev_read_status(b.status) == CODES[code]
    assert torch.isnan(b.out.float()).all()
    for (p, s), (p0, s0) in zip(b.pools, before):
        assert torch.equal(p.view(torch.uint8), p0) and torch.equal(s, s0)


def test_no_tokens_and_no_questions():
    b = Span(103, [0, 0], [5, 0], 4, 2, 128, gaps=2)
    b.chunk()
    b.ok()
    assert (b.out == 0).all()
    b.out.fill_(3.0)
    kev.kev_chunk_attn_paged(b.q, b.k, b.v, 0, b.iv, 2, b.pre, 0, b.cache, 0, 0, b.out, *b.end())
    assert kev.kev_read_status(b.status) == CODES[O.INTERVALS]  # empty, but at tokens 2 and 4 of none
    b.iv.zero_()
    kev.kev_chunk_attn_paged(b.q, b.k, b.v, 0, b.iv, 2, b.pre, 0, b.cache, 0, 0, b.out, *b.end())
    b.ok()
    assert (b.out == 3).all()
    kev.kev_prefill_attn_window(b.q, b.k, b.v, 4, None, 0, 7, 1, b.out, *b.end())
    b.ok()
    assert (b.out[:4] == 0).all()


def test_strided_rows_are_not_needed_but_offset_buffers_are_fine():
    """Buffers that start 16 bytes into an allocation (the alignment the ABI asks for)."""
    b = Span(104, [60, 3], [100, 0], 4, 2, 128)
    ref_in = []
    for name in ("q", "k", "v", "out"):
        x = getattr(b, name)
        y = torch.empty(x.numel() + 8, dtype=x.dtype, device="cuda")[8:].view_as(x)
        y.copy_(x)
        setattr(b, name, y)
        ref_in.append(y.data_ptr() % 32)
    assert 16 in ref_in
    b.chunk(64, 1)
    b.ok()
    b.check(*_kv(b.caches()), 64, 1)


def test_same_bits_alone_in_a_batch_and_again():
    """A question's rows do not depend on its neighbours' values, and calls repeat bit for bit."""
    b = Span(105, [140, 1, 30], [77, 900, 0], 8, 2, 128, "bf16", "e4m3")
    b.chunk(0, 0)
    b.ok()
    one = b.out.clone()
    b.q[140:] = 5.0
    b.out.fill_(float("nan"))
    b.chunk(0, 0)
    b.ok()
    assert torch.equal(one[:140], b.out[:140])


def test_two_streams_and_a_captured_graph():
    """Two calls at once on two streams, each with its own workspace, and a replay after the inputs changed."""
    a, b = (Span(s, [1] * 5, [300, 20, 129, 1000, 0], 8, 2, 128, "bf16", "e4m3") for s in (106, 107))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for x, s in zip((a, b), streams):
            x.chunk(0, 0, max_chunk=1, stream=s)
    torch.cuda.synchronize()
    for x in (a, b):
        x.ok()
        x.check(*_kv(x.caches()), 0, 0)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        a.chunk(256, 4, max_chunk=1)
    a.q.copy_(b.q)
    a.k.copy_(b.k)
    a.prefix = [200, 21, 128, 999, 3]
    a.pre.copy_(torch.tensor(a.prefix, dtype=torch.int32))
    a.out.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    a.ok()
    a.check(*_kv(a.caches()), 256, 4)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_a_prompt_in_pieces_then_decode_equals_the_definition(pool):
    """The operators together, as a serving loop uses them: pieces of prompts, a mixed round and decode steps on one
    cache of a windowed layer; then the cache read back."""
    lens, h_q, h_kv, d, mask = [300, 150], 8, 2, 128, (160, 4)
    total = [m + 3 for m in lens]
    b = Span(108, total, [0, 0], h_q, h_kv, d, "bf16", pool, fill=0.0)
    allq, allk, allv = b.q.clone(), b.k.clone(), b.v.clone()
    start = b.intervals[:, 0].copy()
    out = torch.zeros_like(b.out)
    done = [0, 0]
    for step in ([128, 0], [100, 149], [72, 1], [1, 1], [1, 1], [1, 1]):
        rows = np.concatenate([np.arange(start[i] + done[i], start[i] + done[i] + step[i]) for i in range(2)])
        idx = torch.from_numpy(rows).cuda()
        t = len(rows)
        iv = torch.tensor([[0, step[0]], [step[0], t]], dtype=torch.int32, device="cuda")
        pre = torch.tensor(done, dtype=torch.int32, device="cuda")
        o = torch.empty(t, h_q, d, dtype=torch.bfloat16, device="cuda")
        kev.kev_chunk_attn_paged(allq[idx], allk[idx], allv[idx], t, iv, 2, pre, max(step), b.cache, *mask, o, *b.end())
        b.ok()
        out[idx] = o
        done = [x + y for x, y in zip(done, step)]
    assert done == total
    b.out.copy_(out)
    b.check(*_kv(b.caches()), *mask)
    ko, vo = torch.empty_like(b.k), torch.empty_like(b.v)
    kev.kev_paged_read(ko, vo, b.T, b.iv, 2, b.pre, b.cache, *b.end())
    b.ok()
    if pool == "bf16":
        assert torch.equal(ko, allk) and torch.equal(vo, allv)
    else:
        for got, x in ((ko, allk), (vo, allv)):
            code, sc = O.quantise_rows(x.float().cpu().numpy())
            want = torch.from_numpy(code.astype(np.float32) * sc[..., None]).to(torch.bfloat16)
            assert torch.equal(got.cpu(), want)
    if pool == "bf16":  # one packed prefill of the whole prompts gives the same rows, within both roundings
        b.out.fill_(float("nan"))
        b.packed(*mask)
        b.ok()
        b.check(*_kv(b.caches()), *mask)
