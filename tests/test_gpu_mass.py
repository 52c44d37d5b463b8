"""GPU parity of kev_attn_mass_paged against its float64 definition.

Tolerance.  A score is a sum of d products, off by at most (d + 8) 2^-24 S with S the largest scale sum_e |q_e k_e| of a
visible pair (four times that where the tensor cores add, which keep fewer bits of the smaller terms); a weight is the
exponential of a score less the row's log sum, each off by that, and by a few last places of its argument (at most 2 S in
log2 units) and of the exponential: a relative (8 (d + 8) + 8) S 2^-24 + 2^-20.  A position adds n of them, whose
additions are off by at most n 2^-24 (fewer, as they are added in parts), and decay times the old value, 2^-23 of it.
"""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

import packed_question_isolated_gb300 as kev
from oracle import serve_oracle as S

from test_gpu_span import PAGE, Span

pytestmark = pytest.mark.gpu


class Mass(Span):
    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.bytes = kev.kev_attn_mass_workspace_size(len(self.lens), self.T, self.shape)
        self.ws = torch.full((self.bytes,), 0xff, dtype=torch.uint8, device="cuda")
        g = np.random.default_rng(77)
        self.old = np.exp(g.standard_normal((self.n_blocks, self.h_kv, PAGE))).astype(np.float32)
        self.mass = torch.from_numpy(self.old).cuda()

    def call(self, decay=1.0, max_chunk=0, **kw):
        return kev.kev_attn_mass_paged(self.q, self.T, self.iv, len(self.lens), self.pre, max_chunk, self.cache, decay, self.mass,
                                       *self.end(), **kw)

    def positions(self, x, i):
        n = self.prefix[i] + self.lens[i]
        b = np.maximum(self.table[i, :-(-n // PAGE)], 0)
        return x[b].transpose(0, 2, 1).reshape(-1, self.h_kv)[:n]

    def check(self, decay=1.0, old=None):
        old = self.old if old is None else old
        got = self.mass.cpu().numpy()
        q = self.q.float().cpu().numpy().astype(np.float64)
        live = [i for i in range(len(self.lens)) if self.lens[i]]
        olds = [self.positions(old, i) for i in range(len(self.lens))]
        want, top = S.attn_mass(q, [k for k, _ in self.caches()], self.prefix, self.intervals, olds, decay)
        rel = ((8 * (self.d + 8) + 8) * top + 16 + max(self.lens) * self.h_q / self.h_kv) * 2.0 ** -24
        left = np.ones_like(old, dtype=bool)
        for i in live:
            x, y = self.positions(got, i).astype(np.float64), want[i]
            with np.errstate(invalid="ignore"):
                assert (np.abs(x - y) <= rel * np.abs(y) + 1e-30).all(), (i, np.abs(x / y - 1).max(), rel)
            n = self.prefix[i] + self.lens[i]
            u = np.arange(n)
            left[self.table[i, u // PAGE], :, u % PAGE] = False
        np.testing.assert_array_equal(got[left], old[left])  # nothing else moved


HEADS = [(8, 2), (4, 4), (7, 1), (16, 1), (12, 4), (15, 3)]
DECODE = ([1, 1, 0, 1, 1, 1], [0, 127, 50, 128, 1000, 300])
CHUNK = ([5, 0, 130, 33, 1], [127, 40, 0, 300, 260])


@pytest.mark.parametrize("decay", [1.0, 0.0, 0.75])
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", HEADS)
def test_decode(heads, d, pool, decay):
    m = Mass(1, *DECODE, *heads, d, "bf16", pool)
    m.call(decay, 1)
    m.ok()
    m.check(decay)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", HEADS)
def test_chunks(heads, d, pool):
    m = Mass(2, *CHUNK, *heads, d, "bf16", pool, gaps=1)
    m.call(0.5)
    m.ok()
    m.check(0.5)


@pytest.mark.parametrize("pool", ["fp32", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [DECODE, CHUNK])
def test_fp32(lens, d, pool):
    m = Mass(3, *lens, 6, 2, d, "fp32", pool, gaps=1)
    m.call(1.0, max(lens[0]))
    m.ok()
    m.check()


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 5, 8, 17, 40, 64, 65])
def test_sizes_where_the_kernels_change(tokens, pool):
    for max_chunk in {0, tokens}:
        m = Mass(4, [tokens, 1, tokens], [0, 255, 700], 8, 2, 128, "bf16", pool)
        m.call(1.0, max_chunk)
        m.ok()
        m.check()


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_a_long_cache(pool):
    m = Mass(5, [1, 1], [20000, 5], 4, 1, 128, "bf16", pool)
    m.call(1.0, 1)
    m.ok()
    m.check()


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_a_long_chunk(pool):
    m = Mass(6, [600, 20], [1500, 0], 4, 1, 64, "bf16", pool, order=[1, 0])
    m.call(0.0)
    m.ok()
    m.check(0.0)


@pytest.mark.parametrize("max_chunk", [0, 1])
def test_a_table_far_wider_than_the_caches(max_chunk):
    m = Mass(7, [1, 1], [700, 20], 4, 1, 128, "bf16", "bf16", width=4000)
    m.call(1.0, max_chunk)
    m.ok()
    m.check()


@pytest.mark.parametrize("tokens", [1, 50])
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_what_lies_behind_the_positions_does_not_count(pool, tokens):
    """NaN and infinities in rows and scales behind the last position, stale NaN in the new positions' mass, and V
    anything: the same result, bit for bit."""
    results = []
    for bad in (False, True):
        m = Mass(8, [tokens, tokens], [100, 700 - tokens], 8, 2, 64, "bf16", pool)
        (k, ks), (v, vs) = m.pools
        if bad:
            nan = float("nan")
            v.view(torch.uint8).fill_(0xff)
            for i in range(2):
                n = m.prefix[i] + m.lens[i]
                b = int(m.table[i, (n - 1) // PAGE])
                if pool == "e4m3":
                    k.view(torch.uint8)[b, :, n % PAGE or PAGE:] = 0xff
                    ks[b, :, n % PAGE or PAGE:] = nan
                    ks[b, :, -1] = float("inf") if n % PAGE else ks[b, :, -1]
                else:
                    k[b, :, n % PAGE or PAGE:] = nan
                for u in range(m.prefix[i], n):
                    m.mass[int(m.table[i, u // PAGE]), :, u % PAGE] = nan
        m.call(1.0, tokens)
        m.ok()
        results.append([m.positions(m.mass.cpu().numpy(), i) for i in range(2)])
    for x, y in zip(*results):
        assert np.isfinite(x).all()
        np.testing.assert_array_equal(x, y)


@pytest.mark.parametrize("tokens", [1, 70])
def test_a_nan_reaches_its_own_head_only(tokens):
    m = Mass(9, [tokens, 3], [40, 200], 8, 2, 64, "bf16", "bf16")
    m.q[tokens - 1, 5] = float("nan")  # head 1 of question 0
    m.call(1.0, max(tokens, 3))
    m.ok()
    x = m.positions(m.mass.cpu().numpy(), 0)
    assert np.isnan(x[:, 1]).all() and np.isfinite(x[:, 0]).all()
    assert np.isfinite(m.positions(m.mass.cpu().numpy(), 1)).all()


@pytest.mark.parametrize("tokens,max_chunk", [(1, 1), (40, 0)])
def test_a_scale_of_the_callers_and_large_scores(tokens, max_chunk):
    m = Mass(10, [tokens], [300], 4, 2, 64, "bf16", "bf16")
    m.shape = kev.make_shape(4, 2, 64, "bf16", 2.0)  # scores of up to 100: one position takes nearly all
    m.call(0.0, max_chunk)
    m.ok()
    q = m.q.float().cpu().numpy().astype(np.float64)
    want, top = S.attn_mass(q, [k for k, _ in m.caches()], m.prefix, m.intervals, [m.positions(m.old, 0)], 0, scale=2.0)
    rel = ((8 * 72 + 8) * top + 16 + 2 * tokens) * 2.0 ** -24
    x = m.positions(m.mass.cpu().numpy(), 0)
    assert (np.abs(x - want[0]) <= rel * want[0] + 2.0 ** -120).all()
    assert abs(x.sum() - tokens * 4) < 1e-2


@pytest.mark.parametrize("max_chunk", [0, 3])
def test_device_errors_write_nothing(max_chunk):
    def run(code, change):
        m = Mass(11, [3, 2], [100, 200], 4, 2, 64, "bf16", "bf16")
        change(m)
        m.to_device()
        m.call(1.0, max_chunk, check=True)
        assert kev.kev_read_status(m.status) == getattr(kev.binding, "KEV_ERR_" + code)
        np.testing.assert_array_equal(m.mass.cpu().numpy(), m.old)

    run("INTERVALS", lambda m: m.intervals.__setitem__((1, 0), 0))
    run("PREFIX", lambda m: m.prefix.__setitem__(1, -1))
    run("SLOT_OVERFLOW", lambda m: m.prefix.__setitem__(0, 1 << 20))
    run("SLOT", lambda m: m.table.__setitem__((1, 0), -1))
    run("SLOT", lambda m: m.table.__setitem__((1, 1), int(m.table[0, 0])))


def test_longer_than_announced_is_an_error():
    m = Mass(12, [3, 2], [100, 200], 4, 2, 64, "bf16", "bf16")
    m.call(1.0, 2, check=True)
    assert kev.kev_read_status(m.status) == kev.binding.KEV_ERR_INTERVALS


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_no_tokens(dtype):
    m = Mass(13, [0, 0], [0, 300], 4, 2, 64, dtype, dtype)
    m.call()
    m.ok()
    np.testing.assert_array_equal(m.mass.cpu().numpy(), m.old)


@pytest.mark.parametrize("tokens,max_chunk", [(1, 1), (90, 0)])
def test_the_same_bits_every_time_and_captured(tokens, max_chunk):
    m = Mass(14, [tokens] * 4, [900, 100, 3000, 0], 8, 2, 128, "bf16", "e4m3")
    m.call(0.5, max_chunk)
    m.ok()
    want = m.mass.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            m.call(0.5, max_chunk)
    for _ in range(5):
        m.mass.copy_(torch.from_numpy(m.old))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        m.ok()
        assert (m.mass == want).all()


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHILD = textwrap.dedent(r"""
    import os, sys
    sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]
    from test_gpu_mass import Mass, kev
    for pool in ("bf16", "e4m3"):
        m = Mass(15, [90, 300, 1], [900, 100, 3000], 8, 2, 128, "bf16", pool)
        os.environ.update(KEV_TEST_STALL="1", KEV_TEST_WAIT_LIMIT="2000000")  # ~1 ms
        m.call()
        assert kev.kev_read_status(m.status) == kev.binding.KEV_ERR_TIMEOUT
        del os.environ["KEV_TEST_STALL"], os.environ["KEV_TEST_WAIT_LIMIT"]
        m = Mass(15, [90, 300, 1], [900, 100, 3000], 8, 2, 128, "bf16", pool)
        m.call()
        m.ok()
        m.check()
    print("ALL OK")
""").replace("ROOT", repr(ROOT))


def test_a_wait_that_runs_out_is_reported():
    env = {k: v for k, v in os.environ.items() if k not in ("KEV_TEST_STALL", "KEV_TEST_WAIT_LIMIT")}
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0 and "ALL OK" in r.stdout, f"child failed:\n{r.stdout}\n{r.stderr[-4000:]}"


@pytest.mark.parametrize("tokens,max_chunk", [(1, 1), (70, 0)])
def test_two_calls_at_once_on_two_streams(tokens, max_chunk):
    """Each with a workspace of its own, over one cache, into a mass of its own."""
    a = Mass(16, [tokens] * 3, [700, 0, 2000], 8, 2, 128, "bf16", "bf16")
    b = Mass(16, [tokens] * 3, [700, 0, 2000], 8, 2, 128, "bf16", "bf16")
    b.cache = a.cache
    b.tab, b.table = a.tab, a.table
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for m, s in zip((a, b), streams):
            m.call(0.0, max_chunk, stream=s)
    torch.cuda.synchronize()
    a.ok()
    b.ok()
    a.check(0.0)
    assert (a.mass == b.mass).all()
