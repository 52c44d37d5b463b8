"""GPU parity of kev_norm_rope_paged (norms, rotation, cache write) against its float64 definition.

Tolerances.  A row's sum of d squares is off by at most a relative (d + 2) 2^-24, its mean, eps, the reciprocal root (2
units in the last place) and the two products by (d / 2 + 8) 2^-24 altogether; cos and sin are the table's, rounded to
fp32 (2^-24 of at most 1), and the turned pair is a sum of two products: an output is off by at most (d / 2 + 12) 2^-24
(|a| + |b|), a and b being the pair before the turn.  Rounding to bf16 adds half a step, 2^-8 of the value.  An e4m3 row
comes back off by at most max(2^-4 |y|, 2^-10 s) for the rounding of its codes, beside the fp32 part.
"""
import numpy as np
import pytest
import torch

import packed_question_isolated_gb300 as kev
from oracle import serve_oracle as S

from test_gpu_span import PAGE, TD, Span

pytestmark = pytest.mark.gpu
THETA, EPS = 1e4, 1e-5


class Norm(Span):
    def __init__(self, seed, lens, prefix, h_q, h_kv, d, dtype="bf16", pool="bf16", fused=True, weights=(True, True), start=None, **kw):
        super().__init__(seed, lens, prefix, h_q, h_kv, d, dtype, pool, **kw)
        g = np.random.default_rng(seed + 1)
        self.rows = torch.from_numpy(3 * g.standard_normal((self.T, (h_q + 2 * h_kv) * d), dtype=np.float32)).to(TD[dtype]).cuda()
        cut = [0, h_q * d, (h_q + h_kv) * d, (h_q + 2 * h_kv) * d]
        self.q, self.k, self.v = (self.rows[:, a:b] for a, b in zip(cut, cut[1:]))
        if not fused:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.strides = tuple(x.stride(0) if fused else 0 for x in (self.q, self.k, self.v))
        self.w = [torch.from_numpy(1 + 0.3 * g.standard_normal(d, dtype=np.float32)).to(TD[dtype]).cuda() if on else None for on in weights]
        self.start = list(prefix) if start is None else list(start)
        self.pos = None if start is None else torch.tensor(start, dtype=torch.int32, device="cuda")
        self.max_pos = max([s + m for s, m in zip(self.start, lens)] + [1])
        self.rope = torch.empty(self.max_pos, d // 2, 2, device="cuda")
        kev.kev_rope_table(self.rope, self.max_pos, d, THETA)
        self.q_out = torch.full((self.T, h_q, d), -5.0, dtype=TD[dtype], device="cuda")
        self.k_out = torch.full((self.T, h_kv, d), -6.0, dtype=TD[dtype], device="cuda")

    def call(self, cache=True, k_out=True, max_pos=None, **kw):
        return kev.kev_norm_rope_paged(self.q, self.k, self.v if cache else None, *self.strides, self.q_out,
                                       self.k_out if k_out else None, self.T, self.iv, len(self.lens), self.pre, self.pos, *self.w,
                                       EPS, self.rope, self.max_pos if max_pos is None else max_pos,
                                       self.cache if cache else None, *self.end(), **kw)

    def expect(self):
        """q, k turned, the bound on their error before rounding, and which packed rows belong to a question."""
        live = np.zeros(self.T, bool)
        pos = np.zeros(self.T)
        for (b, e), s in zip(self.intervals, self.start):
            live[b:e] = True
            pos[b:e] = s + np.arange(e - b)
        res = []
        for x, h, w in ((self.q, self.h_q, self.w[0]), (self.k, self.h_kv, self.w[1])):
            x = x.float().cpu().numpy().astype(np.float64).reshape(self.T, h, self.d)
            w = None if w is None else w.float().cpu().numpy()
            y = S.norm_rope(x, w, EPS, np.zeros(self.T), THETA)
            half = np.abs(y[..., :self.d // 2]) + np.abs(y[..., self.d // 2:])
            res.append((S.norm_rope(x, w, EPS, pos, THETA), np.concatenate([half, half], -1) * (self.d / 2 + 12) * 2.0 ** -24))
        return res, live

    def check(self, before, cache=True, k_out=True):
        (q, k), live = self.expect()
        round_off = 0 if self.dtype == "fp32" else 2.0 ** -8

        def near(got, want, more):
            got = got.float().cpu().numpy().astype(np.float64)
            assert (np.abs(got - want[0]) <= want[1] + more * np.abs(want[0]) + 1e-30)[live].all()

        near(self.q_out, q, round_off)
        assert (self.q_out[torch.from_numpy(~live).cuda()] == -5).all() and (self.k_out[torch.from_numpy(~live).cuda()] == -6).all()
        if k_out:
            near(self.k_out, k, round_off)
        else:
            assert (self.k_out == -6).all()
        stored = self.stored()
        if not cache:
            assert all((x == y).all() for x, y in zip(stored, before))
            return
        v = self.v.float().cpu().numpy().astype(np.float64).reshape(self.T, self.h_kv, self.d)
        untouched = np.ones(stored[0].shape[:1] + (PAGE,), bool)
        for i, ((b, e), p) in enumerate(zip(self.intervals, self.prefix)):
            for j in range(e - b):
                blk, row = self.table[i, (p + j) // PAGE], (p + j) % PAGE
                untouched[blk, row] = False
                for side, (y, tol) in enumerate(((k[0][b + j], k[1][b + j]), (v[b + j], 0 * k[1][b + j]))):
                    got = stored[side][blk, :, row]
                    if self.pool == "e4m3":
                        s = np.abs(y).max(-1, keepdims=True) / 448
                        bound = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s) * (1 + 1e-4) + 2 * tol + 1e-30
                    else:
                        bound = tol + (round_off * np.abs(y) if side == 0 else 0) + 1e-30
                    assert (np.abs(got - y) <= bound).all(), (i, j, side)
        for x, y in zip(stored, before):
            assert (x == y).transpose(0, 2, 1, 3)[untouched].all()


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("pool", ["same", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("h_q,h_kv,d", [(8, 2, 128), (7, 1, 64), (16, 16, 64), (28, 4, 128), (1, 1, 128), (30, 2, 64)])
def test_small_calls(h_q, h_kv, d, dtype, pool, fused):
    n = Norm(3, [1, 0, 5, 130, 1], [0, 7, 127, 60, 300], h_q, h_kv, d, dtype, dtype if pool == "same" else pool, fused, gaps=2,
             start=[4, 0, 127, 1000, 301])
    before = n.stored()
    n.call()
    n.ok()
    n.check(before)


@pytest.mark.parametrize("pool,dtype", [("bf16", "bf16"), ("e4m3", "bf16"), ("fp32", "fp32"), ("e4m3", "fp32")])
def test_large_calls(pool, dtype):
    n = Norm(5, [700, 1, 0, 333, 90], [3, 130, 9, 0, 127], 12, 4, 64 if dtype == "fp32" else 128, dtype, pool, gaps=1, order=[3, 0, 4, 1, 2])
    before = n.stored()
    n.call(k_out=False)
    n.ok()
    n.check(before, k_out=False)


@pytest.mark.parametrize("n_questions", [512, 513, 700])
def test_many_questions(n_questions):
    n = Norm(6, [1 if i % 3 else 0 for i in range(n_questions)], [i % 150 for i in range(n_questions)], 4, 2, 64, pool="e4m3")
    before = n.stored()
    n.call()
    n.ok()
    n.check(before)


@pytest.mark.parametrize("T", [40, 600])
@pytest.mark.parametrize("weights", [(False, False), (True, False), (False, True)])
def test_without_norms_and_without_a_cache(weights, T):
    n = Norm(7, [T - 8, 3], [0, 40], 6, 2, 64, weights=weights, gaps=1)
    before = n.stored()
    n.call(cache=False)
    n.ok()
    n.check(before, cache=False)
    n.pre = None  # neither prefixes nor positions: counted from 0
    n.start = [0, 0]
    n.call(cache=False)
    n.ok()
    n.check(before, cache=False)


@pytest.mark.parametrize("T", [40, 600])
def test_in_place_gives_the_same_rows(T):
    n = Norm(8, [T], [9], 6, 2, 128, fused=False)
    n.call()
    n.ok()
    q, k = n.q_out.clone(), n.k_out.clone()
    n.q_out, n.k_out = n.q, n.k
    n.call()
    n.ok()
    assert (n.q.view_as(q) == q).all() and (n.k.view_as(k) == k).all()


def test_rows_of_zeros_and_not_finite_rows():
    n = Norm(9, [4], [0], 2, 1, 64, "bf16", "e4m3")
    n.rows[0] = 0
    n.rows[1, :64] = float("nan")
    n.rows[2, 128:192] = float("inf")  # k
    n.call()
    n.ok()
    assert (n.q_out[0] == 0).all() and (n.k_out[0] == 0).all()
    assert torch.isnan(n.q_out[1, 0]).all() and torch.isfinite(n.q_out[1, 1].float()).all()
    assert torch.isfinite(n.q_out[2:].float()).all()
    stored = n.stored()[0][n.table[0, 0], 0]
    assert (stored[0] == 0).all() and np.isnan(stored[2]).all() and np.isfinite(stored[3]).all()


@pytest.mark.parametrize("T", [6, 600])
def test_device_errors_write_nothing(T):
    def run(code, change, **kw):
        n = Norm(10, [T - 3, 3], [5, 200], 4, 2, 64, pool="e4m3")
        change(n)
        n.to_device()
        before = [x.clone() for pair in n.pools for x in pair]
        n.call(check=True, **kw)
        assert kev.kev_read_status(n.status) == getattr(kev.binding, "KEV_ERR_" + code)
        assert (n.q_out == -5).all() and (n.k_out == -6).all()
        assert all((x.view(torch.uint8) == y.view(torch.uint8)).all() for x, y in zip([x for pair in n.pools for x in pair], before))

    def at(name, *index, value):
        def f(n):
            x = getattr(n, name)
            if len(index) == 1:
                x[index[0]] = value
            else:
                x[index] = value
        return f

    run("INTERVALS", at("intervals", 1, 0, value=0))
    run("INTERVALS", at("intervals", 1, 1, value=T + 1))
    run("PREFIX", at("prefix", 1, value=-1))
    run("SLOT_OVERFLOW", at("prefix", 0, value=1 << 20))
    run("SLOT", at("table", 1, 1, value=-1))
    run("SLOT", lambda n: n.table.__setitem__((1, 1), int(n.table[0, 0])))
    for T0 in (0, 202):
        run("POSITION", lambda n: None, max_pos=T0 or 1)
    run("POSITION", lambda n: setattr(n, "pos", torch.tensor([0, -1], dtype=torch.int32, device="cuda")))
    run("POSITION", lambda n: setattr(n, "pos", torch.tensor([0, 2 ** 31 - 1], dtype=torch.int32, device="cuda")))
    run("SLOT", lambda n: (n.table.__setitem__((1, 1), -1), setattr(n, "pos", torch.tensor([0, -1], dtype=torch.int32, device="cuda"))))


def test_no_tokens():
    n = Norm(11, [0, 0], [0, 3], 4, 2, 64)
    n.call(check=True)
    n.ok()


@pytest.mark.parametrize("T", [32, 700])
def test_captured_on_another_stream(T):
    n = Norm(12, [T - 1, 1], [1, 2], 4, 2, 128, pool="e4m3")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        n.call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            n.call()
    torch.cuda.synchronize()
    want = n.q_out.clone(), n.k_out.clone()
    n.rows *= 2
    for _ in range(2):
        n.q_out.zero_()
        g.replay()
        torch.cuda.synchronize()
        n.ok()
        # the norm undoes the factor, but for eps
        assert torch.allclose(n.q_out.float(), want[0].float(), rtol=2 ** -6, atol=1e-3)
