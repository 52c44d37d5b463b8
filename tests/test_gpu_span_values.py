"""The span operators on values at the ends of their types' ranges, and with a scale of the caller's, against the float64
oracle.

Tolerances, for out = sum_u w_u v_u with weights w_u of sum 1, size = sum_u w_u |v_u|, n positions and
S = scale sum_e |q_e k_e| of the largest key:
* the result is rounded to bf16 once: half a step, 2^-8 of at most size (2^-134 below the normal range);
* the weights are rounded once for the product with V: 2^-8 of each to bf16, so 2^-8 size; to fp16 (decode over e4m3)
  2^-11 size, and for those below fp16's normal range 2^-25 per position of the unit that they are held in: the largest
  w_u s_u so far, s_u = max_e |v_ue| / 448, or 2^-126 if that is more; codes are at most 448;
* fp32: a score is off by (d + 2) 2^-24 S, so a weight by a relative (d + 8) 2^-24 S + 2^-21, both in the sum of the
  weights and in the sum over v, and the sums by (n + 4) 2^-24: (2 (d + 8) S + 2 n + 32) 2^-24 size;
* exponentials below 2^-126 are zero: 2^-126 sum_u |v_u|.
"""
import numpy as np
import pytest
import torch

import packed_question_isolated_gb300 as kev
from oracle import kev_oracle as O

from test_gpu_span import PAGE, Span

pytestmark = pytest.mark.gpu


def against_oracle(b, caches, mask=(0, 0), scale=None, weights=2.0 ** -8, rows=None):
    """b.out against the oracle over `caches`; `weights`: half a step of the softmax weights' type; `rows`: the tokens looked at."""
    q = b.q.float().cpu().numpy().astype(np.float64)
    got = b.out.float().cpu().numpy().astype(np.float64)
    sc = 1 / np.sqrt(b.d) if scale is None else scale
    worst = 0.0
    for i, (s, e) in enumerate(b.intervals):
        k, v = caches[i]
        for t in range(s, e):
            if rows is not None and t not in rows:
                continue
            p = b.prefix[i] + t - s
            seen = O.span_visible(p, p + 1, *mask)
            for h in range(b.h_q):
                g = h // (b.h_q // b.h_kv)
                ku, vu = k[:p + 1, g][seen], v[:p + 1, g][seen]
                z = sc * (ku @ q[t, h])
                w = np.exp(z - z.max())
                w /= w.sum()
                n, ref, size = len(z), w @ vu, w @ np.abs(vu)
                big = sc * (np.abs(ku) @ np.abs(q[t, h])).max()
                tol = (2 * (b.d + 8) * big + 2 * n + 32) * 2.0 ** -24 * size + 2.0 ** -126 * np.abs(vu).sum(0)
                if b.dtype == "bf16":
                    tol += (2.0 ** -8 + weights) * size + 2.0 ** -134
                    if weights < 2.0 ** -8:
                        tol += n * 2.0 ** -25 * max((w * np.abs(vu).max(-1)).max(), 448 * 2.0 ** -126)
                err = np.abs(got[t, h] - ref)
                assert (err <= tol).all(), (t, h, float(err.max()), float(tol[err.argmax()]), got[t, h][:4], ref[:4])
                worst = max(worst, float((err / tol).max()))
    return worst


def with_scale(b, scale):
    if scale is not None:
        b.shape = kev.make_shape(b.h_q, b.h_kv, b.d, b.dtype, scale)
    return b


def seen_by_some(b, mask):
    """bool[n_blocks, PAGE]: cached positions that some new token sees."""
    keep = np.zeros((b.n_blocks, PAGE), bool)
    for i, (m, p) in enumerate(zip(b.lens, b.prefix)):
        for x in range(p, p + m):
            for u in np.flatnonzero(O.span_visible(x, x + 1, *mask)):
                keep[b.table[i, u // PAGE], u % PAGE] = True
    return torch.from_numpy(keep).cuda()


# lens, prefix, mask, max_chunk: decode, few rows, chunks, a mixed round
BATCHES = [([1, 1, 1], [300, 129, 5], (100, 2), 1), ([2, 1], [300, 129], (0, 0), 2), ([40, 1, 150], [300, 129, 5], (100, 2), 0),
           ([1] * 12 + [70], [30 * i for i in range(13)], (0, 0), 0)]


def masked_scales(side, bits, batch, dtype, d, scale):
    lens, prefix, mask, mc = BATCHES[batch]
    b = with_scale(Span(400 + batch, lens, prefix, 8, 2, d, dtype, "e4m3"), scale)
    b.write()
    caches = b.caches()
    masked = (~seen_by_some(b, mask))[:, None, :].expand(-1, b.h_kv, -1)
    p, s = b.pools[side]
    s.view(torch.int32)[masked] = int(np.array([bits], np.uint32).view(np.int32)[0])
    g = torch.Generator(device="cuda").manual_seed(bits & 0xffff)
    p.view(torch.uint8)[masked] = torch.randint(0, 256, (int(masked.sum()), d), generator=g, device="cuda", dtype=torch.uint8)
    b.chunk(*mask, max_chunk=mc, write=False)
    b.ok()
    against_oracle(b, caches, mask, scale)


# the smallest subnormals (as small integers look in memory that held some), a product with the scale that underflows,
# -0, infinities, NaN, the largest and the smallest finite number
BITS = [0x1, 0x2, 0x3, 0x400, 0x80000000, 0x80000001, 0xff800000, 0x7f800000, 0xffc00000, 0x7fffffff, 0x7f7fffff, 0xff7fffff]


@pytest.mark.parametrize("bits", BITS, ids=hex)
@pytest.mark.parametrize("batch", range(len(BATCHES)))
@pytest.mark.parametrize("dtype,d,scale", [("bf16", 128, None), ("bf16", 64, 2.0 ** -12), ("fp32", 64, None)])
def test_key_scales_of_masked_positions_may_hold_anything(bits, batch, dtype, d, scale):
    masked_scales(0, bits, batch, dtype, d, scale)


@pytest.mark.parametrize("bits", BITS, ids=hex)
@pytest.mark.parametrize("batch", range(len(BATCHES)))
@pytest.mark.parametrize("dtype,d,scale", [("bf16", 128, None), ("bf16", 64, 2.0 ** -12), ("fp32", 64, None)])
def test_value_scales_of_masked_positions_may_hold_anything(bits, batch, dtype, d, scale):
    masked_scales(1, bits, batch, dtype, d, scale)


def set_value_rows(b, at, factor):
    """Multiplies the cached V rows of positions `at` of every question by `factor`, as quantised rows are: their codes stay."""
    pv, sv = b.pools[1]
    for i, (m, p) in enumerate(zip(b.lens, b.prefix)):
        for u in at(p + m):
            blk, r = int(b.table[i, u // PAGE]), u % PAGE
            if sv is None:
                pv[blk, :, r] *= factor
            else:
                sv[blk, :, r] *= factor


WHERE = [lambda n: range(n), lambda n: range(min(n, PAGE)), lambda n: range(n - n // 3, n), lambda n: range(0, n, 5)]


@pytest.mark.parametrize("factor", [0.0, 1e-43, 1e-40, 1e-37, 1e-35, 1e-33, 1e25])
@pytest.mark.parametrize("where", range(len(WHERE)), ids=["all", "first page", "last", "every fifth"])
@pytest.mark.parametrize("pool,h_q,h_kv,d", [("e4m3", 8, 2, 128), ("e4m3", 16, 1, 64), ("e4m3", 4, 4, 64), ("bf16", 8, 2, 128)])
def test_decode_over_values_of_any_size(pool, h_q, h_kv, d, where, factor):
    b = Span(410, [1, 1, 1], [600, 200, 17], h_q, h_kv, d, "bf16", pool)
    b.write()
    set_value_rows(b, WHERE[where], factor)
    b.chunk(max_chunk=1, write=False)
    b.ok()
    against_oracle(b, b.caches(), weights=2.0 ** -11 if pool == "e4m3" else 2.0 ** -8)


@pytest.mark.parametrize("above", [20, 90, 110, 114, 116, 118, 120, 122, 124, 126, 130, 150, 200])
@pytest.mark.parametrize("key", [0, 3, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_a_key_far_above_the_others_whose_values_are_zero(d, key, above):
    """A null sink: one key's score stands 2^above over the others' and its V row is zero, so the result is the others' share."""
    b = Span(411, [1], [400], 4, 2, d, "bf16", "e4m3")
    b.write()
    (pk, sk), (pv, sv) = b.pools
    b.q.fill_(1.0)
    blk, r = int(b.table[0, key // PAGE]), key % PAGE
    sk.zero_()
    pk.view(torch.uint8).zero_()
    pk.view(torch.uint8)[blk, :, r] = 0x7e  # 448
    sk[blk, :, r] = above * np.log(2.0) / (448 * np.sqrt(d))
    pv.view(torch.uint8)[blk, :, r] = 0
    sv[blk, :, r] = 0.0
    b.chunk(max_chunk=1, write=False)
    b.ok()
    against_oracle(b, b.caches(), weights=2.0 ** -11)


@pytest.mark.parametrize("factor", [0.0, 1e-43, 1e-40, 1e-37, 1e-35, 1e-33, 1e25])
@pytest.mark.parametrize("where", range(len(WHERE)), ids=["all", "first page", "last", "every fifth"])
@pytest.mark.parametrize("pool,d", [("e4m3", 128), ("e4m3", 64), ("bf16", 128)])
def test_chunks_over_values_of_any_size(pool, d, where, factor):
    b = Span(412, [20, 40], [300, 17], 8, 2, d, "bf16", pool)
    b.write()
    set_value_rows(b, WHERE[where], factor)
    b.chunk(write=False)
    b.ok()
    against_oracle(b, b.caches())


@pytest.mark.parametrize("above", [20, 60, 90, 110, 118, 122, 126, 150])
@pytest.mark.parametrize("key", [0, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_chunks_with_a_key_far_above_the_others_whose_values_are_zero(d, key, above):
    b = Span(413, [20], [400], 4, 2, d, "bf16", "e4m3")
    b.write()
    (pk, sk), (pv, sv) = b.pools
    b.q.fill_(1.0)
    blk, r = int(b.table[0, key // PAGE]), key % PAGE
    sk.zero_()
    pk.view(torch.uint8).zero_()
    pk.view(torch.uint8)[blk, :, r] = 0x7e  # 448
    sk[blk, :, r] = above * np.log(2.0) / (448 * np.sqrt(d))
    pv.view(torch.uint8)[blk, :, r] = 0
    sv[blk, :, r] = 0.0
    b.chunk(write=False)
    b.ok()
    against_oracle(b, b.caches())


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("h_q,h_kv", [(16, 1), (12, 1), (9, 1), (8, 2), (4, 4)])
def test_calls_without_tokens(h_q, h_kv, pool):
    """Every question dropped: the checks run, nothing is written, with and without max_chunk."""
    b = Span(420, [0, 0, 0], [700, 3, 0], h_q, h_kv, 128, "bf16", pool, width=6)
    before = [(p.view(torch.uint8).clone(), None if s is None else s.clone()) for p, s in b.pools]
    for mask in ((0, 0), (9, 2)):
        for mc in (0, 1):
            b.status.fill_(-1)
            b.chunk(*mask, max_chunk=mc)
            b.ok()
            assert kev.kev_launch_count(18) == 1
        b.status.fill_(-1)
        b.packed(*mask)
        b.ok()
    for (p, s), (p0, s0) in zip(b.pools, before):
        assert torch.equal(p.view(torch.uint8), p0) and (s is None or torch.equal(s, s0))


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [0, 5, 600])
def test_calls_without_questions(T, pool):
    """Tokens of no question: rows of out are zero, nothing else is touched."""
    b = Span(421, [T], [200], 4, 2, 128, "bf16", pool)
    before = [(p.view(torch.uint8).clone(), None if s is None else s.clone()) for p, s in b.pools]
    ko, vo = b.k.clone(), b.v.clone()
    for f in (kev.kev_paged_write, kev.kev_paged_read):
        b.status.fill_(-1)
        f(ko, vo, T, None, 0, None, b.cache, *b.end())
        b.ok()
    assert torch.equal(ko, b.k) and torch.equal(vo, b.v)
    for mask, mc in (((0, 0), 0), ((9, 2), 0), ((0, 0), 1)):
        b.status.fill_(-1)
        b.out.fill_(3.0)
        kev.kev_chunk_attn_paged(b.q, b.k, b.v, T, None, 0, None, mc, b.cache, *mask, b.out, *b.end())
        b.ok()
        assert (b.out == 0).all()
    for (p, s), (p0, s0) in zip(b.pools, before):
        assert torch.equal(p.view(torch.uint8), p0) and (s is None or torch.equal(s, s0))


@pytest.mark.parametrize("pool", ["packed", "bf16", "e4m3"])
@pytest.mark.parametrize("long,short", [(60, 9), (40, 30), (64, 64)])
def test_infinities_are_put_back_in_every_unit(pool, long, short):
    """Many units per CTA, of two row tiles and of one in turns, each with an infinity (e4m3: a NaN row) in the middle of its V:
    the rows that see it get it, the others are as without it."""
    h_q, h_kv, d, n = 16, 4, 64, 600
    r = np.random.default_rng(430 + long)
    lens = np.where(r.random(n) < 0.5, long, short) - r.integers(0, 8, n)
    b = Span(430, lens.tolist(), [0] * n, h_q, h_kv, d, "bf16", "bf16" if pool == "packed" else pool)
    at = torch.from_numpy(b.intervals[:, 0] + (lens * 0.6).astype(int)).cuda()
    if pool == "packed":
        b.v[at, :, 5::17] = float("inf")
        b.packed(0, 0)
    else:
        b.write()
        blk = torch.from_numpy(b.table[:, 0]).cuda().long()
        row = at - b.iv[:, 0]
        pv, sv = b.pools[1]
        if pool == "bf16":
            pv[blk, :, row, 5::17] = float("inf")
        else:
            pv.view(torch.uint8)[blk, :, row] = 0x7f
            sv[blk, :, row] = float("nan")
        b.chunk(write=False)
    b.ok()
    stored = [torch.from_numpy(x).cuda() for x in b.stored()] if pool != "packed" else None
    for i, (s, e) in enumerate(b.intervals.tolist()):
        if pool == "packed":
            k, v = b.k[s:e].double(), b.v[s:e].double()
        else:
            k, v = (x[int(b.table[i, 0])].transpose(0, 1)[:e - s] for x in stored)
        q = b.q[s:e].double().view(e - s, h_kv, h_q // h_kv, d)
        z = torch.einsum("thgd,uhd->thgu", q, k) / 8
        seen = torch.ones(e - s, e - s, dtype=torch.bool, device="cuda").tril()[:, None, None]
        w = torch.softmax(z.masked_fill(~seen, -np.inf), -1)
        ok = v.isfinite()
        clean = torch.where(ok, v, 0)
        ref, size = (torch.einsum("thgu,uhd->thgd", w, x).reshape(e - s, h_q, d) for x in (clean, clean.abs()))
        hit = torch.einsum("thgu,uhd->thgd", seen.expand_as(z).double(), (~ok).double()).reshape(e - s, h_q, d) > 0
        got = b.out[s:e].double()
        assert torch.equal(~got.isfinite(), hit), i
        # two roundings to bf16 and the fp32 part: scores of at most a few tens
        assert ((got - ref).abs() <= (2.0 ** -7 + 2.0 ** -12) * size + 1e-30)[~hit].all(), i


@pytest.mark.parametrize("what", ["prefix", "overflow", "range", "twice"])
@pytest.mark.parametrize("more", [0, 600])
def test_overlapping_intervals_come_before_other_errors(what, more):
    """Of several errors the first in the order intervals, prefix, overflow, slot is reported, whatever question has it."""
    b = Span(431, [5, 9, 4], [130, 40, 0], 4, 2, 128, "bf16", "e4m3")
    b.intervals[2] = (2, 3)  # inside question 0
    if what == "prefix":
        b.prefix[1] = -1
    elif what == "overflow":
        b.prefix[1] = b.width * PAGE - 8
    elif what == "range":
        b.table[0, 1] = b.n_blocks
    else:
        b.table[1, 0] = b.table[0, 1]
    b.to_device()
    assert O.validate_span(b.intervals, b.T + more, b.prefix, b.table, b.n_blocks) == O.INTERVALS
    want = kev.binding.KEV_ERR_INTERVALS
    T = b.T + more
    q, k, v, out = (torch.cat([x, torch.ones((more, *x.shape[1:]), dtype=x.dtype, device="cuda")]) for x in (b.q, b.k, b.v, b.out))
    ws = torch.full((kev.kev_paged_workspace_size(3, T, b.shape),), 0xff, dtype=torch.uint8, device="cuda")
    end = (b.shape, ws, ws.numel(), b.status)
    before = [(p.view(torch.uint8).clone(), s.clone()) for p, s in b.pools]
    for f in (kev.kev_paged_write, kev.kev_paged_read):
        b.status.fill_(-1)
        f(k, v, T, b.iv, 3, b.pre, b.cache, *end)
        assert kev.kev_read_status(b.status) == want
    b.status.fill_(-1)
    kev.kev_chunk_attn_paged(q, k, v, T, b.iv, 3, b.pre, 0, b.cache, 0, 0, out, *end)
    assert kev.kev_read_status(b.status) == want
    for (p, s), (p0, s0) in zip(b.pools, before):
        assert torch.equal(p.view(torch.uint8), p0) and torch.equal(s, s0)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 128), ("fp32", 64)])
@pytest.mark.parametrize("how", ["small", "large", "decode"])
def test_rows_with_subnormal_scales_are_written_as_defined(dtype, d, how):
    """Rows of 2^-149 to 2^-100 and of the largest numbers: codes and scales bit for bit, by both copies and by a decode step."""
    n, h_kv = (300, 3) if how == "large" else (120, 3)
    b = Span(440, [1] * n if how == "decode" else [n], list(range(n)) if how == "decode" else [70], 6, h_kv, d, dtype, "e4m3")
    g = torch.Generator(device="cuda").manual_seed(440)
    for x in (b.k, b.v):
        e = torch.randint(-149, -99, (n, h_kv, 1), generator=g, device="cuda")
        e[::7] = 126
        x.copy_(torch.ldexp(x.double(), e).clamp(-3.3e38, 3.3e38).to(x.dtype))
    if how == "decode":
        b.chunk(max_chunk=1)
    else:
        k, v = (torch.cat([x, torch.zeros((500 if how == "large" else 0, h_kv, d), dtype=x.dtype, device="cuda")]) for x in (b.k, b.v))
        ws = torch.empty(kev.kev_paged_workspace_size(1, len(k), b.shape), dtype=torch.uint8, device="cuda")
        kev.kev_paged_write(k, v, len(k), b.iv, 1, b.pre, b.cache, b.shape, ws, ws.numel(), b.status)
    b.ok()
    t = np.arange(n)
    q, pos = (t, np.array(b.prefix)) if how == "decode" else (np.zeros(n, int), 70 + t)
    row = b.intervals[q, 0] + (0 if how == "decode" else t)
    blk = b.table[q, pos // PAGE]
    for x, (p, s) in zip((b.k, b.v), b.pools):
        code, scale = O.quantise_rows(x.float().cpu().numpy()[row])
        want = torch.from_numpy(code).float().to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(s.cpu()[blk, :, pos % PAGE], torch.from_numpy(scale))
        assert torch.equal(p.view(torch.uint8).cpu()[blk, :, pos % PAGE], want)


@pytest.mark.parametrize("shift", [-124, -118, -110, -100, -60, 60, 100])
@pytest.mark.parametrize("dtype,pool,d", [("bf16", "e4m3", 128), ("bf16", "e4m3", 64), ("bf16", "bf16", 128), ("fp32", "e4m3", 64)])
@pytest.mark.parametrize("lens,max_chunk", [([1, 1], 1), ([2, 1], 2), ([20, 40], 0)])
def test_small_q_and_large_k_and_the_other_way_round(lens, max_chunk, dtype, pool, d, shift):
    """Rows of q times 2^shift, cached K times 2^-shift: the scores are as without either."""
    b = Span(450, lens, [300, 17], 8, 2, d, dtype, pool)
    b.write()
    b.q.copy_(torch.ldexp(b.q.double(), torch.tensor(shift, device="cuda")).to(b.q.dtype))
    pk, sk = b.pools[0]
    x = pk if sk is None else sk
    x.copy_(torch.ldexp(x.double(), torch.tensor(-shift, device="cuda")).to(x.dtype))
    b.chunk(max_chunk=max_chunk, write=False)
    b.ok()
    against_oracle(b, b.caches(), weights=2.0 ** -11 if (dtype, pool) == ("bf16", "e4m3") and max_chunk else 2.0 ** -8)


@pytest.mark.parametrize("side", ["k", "v", "q"])
@pytest.mark.parametrize("dtype,pool", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32"), ("fp32", "e4m3")])
@pytest.mark.parametrize("lens,prefix,max_chunk", [([1, 1, 1], [300, 129, 5], 1), ([2, 1, 2], [300, 129, 126], 2),
                                                   ([40, 1, 150], [300, 129, 5], 0), ([1] * 20 + [70], [9 * i for i in range(21)], 0)])
def test_rows_that_see_a_nan_are_nan_and_no_others(lens, prefix, max_chunk, dtype, pool, side):
    """NaN in a new row of q, k or v (through the cache it goes into) and, for k and v, in a cached one."""
    b = Span(460, lens, prefix, 8, 2, 128, dtype, pool)
    b.write()
    bad = int(b.intervals[-1, 0]) + lens[-1] // 2  # a token of the last question
    at = prefix[-1] + lens[-1] // 2
    if side == "q":
        b.q[bad, 3] = float("nan")
    else:
        x = b.k if side == "k" else b.v
        x[bad, 1] = float("nan")
        p, s = b.pools["kv".index(side)]  # and position 3 of question 0, head 0
        if s is None:
            p[b.table[0, 0], 0, 3] = float("nan")
        else:
            p.view(torch.uint8)[b.table[0, 0], 0, 3] = 0x7f
            s[b.table[0, 0], 0, 3] = float("nan")
    b.chunk(max_chunk=max_chunk)
    b.ok()
    nan = torch.isnan(b.out.float()).cpu().numpy()
    want = np.zeros(nan.shape, bool)
    if side == "q":
        want[bad, 3] = True
    else:
        s0, e0 = b.intervals[0]
        want[[t for t in range(s0, e0) if prefix[0] + t - s0 >= 3], :4] = True
        s1, e1 = b.intervals[-1]
        want[[t for t in range(s1, e1) if prefix[-1] + t - s1 >= at], 4:] = True
    assert (nan == want).all(), np.argwhere(nan != want)[:5]
    assert np.isfinite(b.out.float().cpu().numpy()[~want]).all()
