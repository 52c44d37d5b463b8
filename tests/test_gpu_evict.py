"""GPU parity of kev_select_paged and kev_compact_paged: choices and copies, so everything is equal."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

import packed_question_isolated_gb300 as kev
from oracle import serve_oracle as S

pytestmark = pytest.mark.gpu
PAGE = 128
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Cut:
    def __init__(self, seed, lens, keep, first=0, last=0, h_kv=2, d=64, pool="bf16", width=None, spare=3, mass=True, ties=0):
        g = np.random.default_rng(seed)
        self.lens, self.keep, self.first, self.last, self.h_kv, self.d, self.pool = list(lens), keep, first, last, h_kv, d, pool
        n = len(lens)
        pages = [-(-m // PAGE) for m in lens]
        self.n_blocks, self.width = sum(pages) + spare, width or max(max(pages), 1)
        ids, at = g.permutation(self.n_blocks), 0
        self.table = np.full((n, self.width), -1, np.int32)
        for i, m in enumerate(pages):
            self.table[i, :m] = ids[at:at + m]
            at += m
        shape = (self.n_blocks, h_kv, PAGE)
        m = np.exp(2 * g.standard_normal(shape)).astype(np.float32)
        self.mass = np.floor(m * ties).astype(np.float32) if ties else m
        item = {"bf16": 2, "fp32": 4, "e4m3": 1}[pool]
        self.k, self.v = (g.integers(0, 256, shape + (d * item,), dtype=np.uint8) for _ in range(2))
        self.sk, self.sv = (g.random(shape, dtype=np.float32) for _ in range(2))
        self.shape = kev.make_shape(h_kv * 2, h_kv, d, "fp32" if pool == "fp32" else "bf16")
        self.bytes = kev.kev_evict_workspace_size(n, keep, self.shape)
        self.ws = torch.full((self.bytes,), 0xff, dtype=torch.uint8, device="cuda")
        self.status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        self.kept = np.full((n, h_kv, keep), -9, np.int32)
        self.kept_lens = np.full(n, -9, np.int32)
        self.active = None
        self.with_mass = mass
        self.to_device()

    def to_device(self):
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        self.d_lens, self.d_table, self.d_mass = dev(np.asarray(self.lens, np.int32)), dev(self.table), dev(self.mass)
        self.d_k, self.d_v, self.d_sk, self.d_sv = dev(self.k), dev(self.v), dev(self.sk), dev(self.sv)
        self.d_kept, self.d_kept_lens = dev(self.kept), dev(self.kept_lens)
        self.d_active = None if self.active is None else dev(np.asarray(self.active, np.uint8))
        e4m3 = self.pool == "e4m3"
        self.cache = kev.make_paged_cache(self.d_k, self.d_v, self.d_table, self.width, self.n_blocks, self.pool,
                                          self.d_sk if e4m3 else None, self.d_sv if e4m3 else None)

    def end(self):
        return self.shape, self.ws, self.bytes, self.status

    def select(self, **kw):
        return kev.kev_select_paged(self.d_mass, self.d_lens, self.d_active, len(self.lens), self.d_table, self.width, self.n_blocks,
                                    self.keep, self.first, self.last, self.d_kept, self.d_kept_lens, *self.end(), **kw)

    def compact(self, **kw):
        return kev.kev_compact_paged(self.d_kept, self.keep, self.d_lens, self.d_kept_lens, len(self.lens), self.cache,
                                     self.d_mass if self.with_mass else None, *self.end(), **kw)

    def ok(self):
        assert kev.kev_read_status(self.status) == 0

    def rows(self, x, i, n):
        """Positions 0 .. n - 1 of question i: [n, h_kv, ...]."""
        b = self.table[i, :-(-n // PAGE)]
        return np.moveaxis(x[b], 1, 2).reshape((-1, self.h_kv) + x.shape[3:])[:n]

    def check_select(self):
        kept, kept_lens = self.d_kept.cpu().numpy(), self.d_kept_lens.cpu().numpy()
        for i, n in enumerate(self.lens):
            if self.active is not None and not self.active[i]:
                assert kept_lens[i] == n and (kept[i] == -9).all()
                continue
            want = S.select(self.rows(self.mass, i, n).reshape(n, self.h_kv), self.keep, self.first, self.last)
            assert kept_lens[i] == want.shape[1]
            np.testing.assert_array_equal(kept[i, :, :want.shape[1]], want)
            assert (kept[i, :, want.shape[1]:] == -9).all()

    def state(self):
        return [x.cpu().numpy() for x in (self.d_k, self.d_v, self.d_sk, self.d_sv, self.d_mass)]

    def check_compact(self, kept, kept_lens):
        after = self.state()
        for j, (x, y) in enumerate(zip((self.k, self.v, self.sk, self.sv, self.mass), after)):
            want = x.copy()
            free = np.zeros((self.n_blocks, PAGE), bool)  # rows that hold nothing of use afterwards
            moved = (True, True, self.pool == "e4m3", self.pool == "e4m3", self.with_mass)[j]
            for i, (n, m) in enumerate(zip(self.lens, kept_lens)):
                if m == n:
                    continue
                for u in range(m, n):
                    free[self.table[i, u // PAGE], u % PAGE] = True
                if moved:
                    for g in range(self.h_kv):
                        src, dst = kept[i, g, :m], np.arange(m)
                        want[self.table[i, dst // PAGE], g, dst % PAGE] = x[self.table[i, src // PAGE], g, src % PAGE]
            used = ~free
            same = (np.moveaxis(want, 1, 2) == np.moveaxis(y, 1, 2))
            assert same[used].all(), j


LENS = [[1], [130, 0, 5, 700, 64, 65], [128, 129, 256, 1000]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("keep,first,last", [(1, 0, 0), (64, 4, 16), (65, 0, 65), (100, 100, 0), (129, 1, 3), (300, 4, 0)])
@pytest.mark.parametrize("ties", [0, 1, 3])
def test_select(lens, keep, first, last, ties):
    c = Cut(1, lens, keep, first, last, ties=ties)
    c.select()
    c.ok()
    c.check_select()


@pytest.mark.parametrize("n,keep", [(4096, 1000), (4097, 17), (20000, 4096), (60000, 20000), (60000, 59999)])
@pytest.mark.parametrize("ties", [0, 2])
def test_select_long(n, keep, ties):
    c = Cut(2, [n, n // 3], keep, 4, min(128, keep - 4), h_kv=1, ties=ties)
    c.select()
    c.ok()
    c.check_select()


def test_select_of_a_wide_table():
    """More pages in the table than positions: the kernel for long caches on short ones."""
    c = Cut(3, [300, 40, 1000], 100, 1, 30, width=600)
    c.select()
    c.ok()
    c.check_select()


def test_select_of_odd_masses():
    """NaN above all, infinities, -0 and 0 equal, negative numbers, subnormals; stale NaN outside the cached positions."""
    c = Cut(4, [700, 300], 90, 2, 5)
    g = np.random.default_rng(0)
    flat = c.mass.reshape(-1)
    for value in (np.nan, np.inf, -np.inf, -0.0, 0.0, -1.5, 1e-40, -1e-40):
        flat[g.integers(0, flat.size, flat.size // 12)] = value
    flat[g.integers(0, flat.size, 3)] = np.uint32(0xffc00001).view(np.float32)
    c.to_device()
    c.select()
    c.ok()
    c.check_select()
    c.mass[:] = 0
    c.to_device()
    c.select()
    c.check_select()


def test_select_of_live_questions_only():
    c = Cut(5, [500, 200, 300], 100, 0, 10)
    c.active = [1, 0, 1]
    c.table[1, 1] = 10 ** 6  # not looked at
    c.to_device()
    c.select()
    c.ok()
    c.check_select()


@pytest.mark.parametrize("code,change", [
    ("SLOT_OVERFLOW", lambda c: c.lens.__setitem__(1, -1)), ("SLOT_OVERFLOW", lambda c: c.lens.__setitem__(0, c.width * PAGE + 1)),
    ("SLOT", lambda c: c.table.__setitem__((2, 1), -1)), ("SLOT", lambda c: c.table.__setitem__((2, 1), c.n_blocks))])
def test_select_errors_write_nothing(code, change):
    c = Cut(6, [500, 100, 200], 64)
    change(c)
    c.to_device()
    c.select(check=True)
    assert kev.kev_read_status(c.status) == getattr(kev.binding, "KEV_ERR_" + code)
    assert (c.d_kept == -9).all() and (c.d_kept_lens == -9).all()


@pytest.mark.parametrize("pool", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("keep", [1, 63, 64, 200, 513])
@pytest.mark.parametrize("mass", [True, False])
def test_compact(keep, d, pool, mass):
    c = Cut(7, [1000, 0, 200, 64, 513, 700], keep, min(2, keep), 0, d=d, pool=pool, mass=mass)
    c.select()
    c.ok()
    kept, kept_lens = c.d_kept.cpu().numpy(), c.d_kept_lens.cpu().numpy()
    c.compact()
    c.ok()
    c.check_compact(kept, kept_lens)


@pytest.mark.parametrize("shape", ["tail", "every other", "head", "random", "nothing"])
@pytest.mark.parametrize("n", [5000, 300])
def test_compact_of_lists_of_the_callers(shape, n):
    """Rows that travel far, short ways, not at all; run often, so that chunks meet in every order."""
    m = 0 if shape == "nothing" else n // 2
    c = Cut(8, [n, n - 10, 77], max(m, 77), h_kv=3, pool="e4m3")
    g = np.random.default_rng(1)
    for i, size in enumerate(c.lens[:2]):
        for h in range(3):
            u = {"tail": np.arange(size - m, size), "every other": np.arange(m) * 2 - (i if m * 2 > size else 0), "head": np.arange(m),
                 "random": np.sort(g.permutation(size)[:m]), "nothing": np.arange(0)}[shape]
            if shape == "every other":
                u = np.minimum(u, size - m + np.arange(m))
                u = np.maximum.accumulate(np.maximum(u, np.arange(m)))
                u = np.sort(g.permutation(size)[:m]) if (np.diff(u) <= 0).any() else u
            c.kept[i, h, :m] = u
    c.kept_lens[:] = [m, m, 77]
    for _ in range(5):
        c.to_device()
        c.compact()
        c.ok()
        c.check_compact(c.kept, c.kept_lens)


@pytest.mark.parametrize("code,change", [
    ("KEPT", lambda c: c.kept.__setitem__((0, 1, 5), c.kept[0, 1, 4])), ("KEPT", lambda c: c.kept.__setitem__((2, 0, 63), 200)),
    ("KEPT", lambda c: c.kept.__setitem__((0, 0, 0), -1)), ("KEPT", lambda c: c.kept_lens.__setitem__(0, -1)),
    ("KEPT", lambda c: c.kept_lens.__setitem__(1, 101)), ("KEPT", lambda c: c.kept_lens.__setitem__(2, 65)),
    ("SLOT_OVERFLOW", lambda c: c.lens.__setitem__(1, -1)), ("SLOT_OVERFLOW", lambda c: c.lens.__setitem__(0, c.width * PAGE + 1)),
    ("SLOT", lambda c: c.table.__setitem__((2, 1), -1)), ("SLOT", lambda c: c.table.__setitem__((2, 1), c.n_blocks)),
    ("SLOT", lambda c: c.table.__setitem__((2, 0), c.table[0, 1])),
    ("SLOT", lambda c: (c.table.__setitem__((2, 0), c.table[0, 1]), c.kept.__setitem__((0, 0, 0), -1)))])
def test_compact_errors_write_nothing(code, change):
    c = Cut(9, [500, 100, 200], 64)
    c.kept[:] = np.arange(64) + 3
    c.kept_lens[:] = 64
    change(c)
    c.to_device()
    c.compact(check=True)
    assert kev.kev_read_status(c.status) == getattr(kev.binding, "KEV_ERR_" + code)
    assert all((x == y).all() for x, y in zip(c.state(), (c.k, c.v, c.sk, c.sv, c.mass)))


def test_questions_that_are_not_cut_are_not_looked_at():
    c = Cut(10, [500, 100, 200], 64)
    c.kept[:] = np.arange(64) + 3
    c.kept_lens[:] = [64, 100, 200]
    c.kept[1:] = -1
    c.table[2] = -5
    c.to_device()
    c.compact()
    c.ok()
    c.table[2] = 0
    c.check_compact(c.kept, c.kept_lens)


def test_two_streams_and_a_captured_graph():
    a, b = Cut(11, [3000, 2000], 700, 4, 30, pool="e4m3"), Cut(12, [4000, 100], 900, 4, 30)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for c, st in zip((a, b), s):
        with torch.cuda.stream(st):
            c.select(stream=st)
            c.compact(stream=st)
    torch.cuda.synchronize()
    for c in (a, b):
        c.ok()
        c.check_select()
        c.check_compact(c.d_kept.cpu().numpy(), c.d_kept_lens.cpu().numpy())
    start = [x.clone() for x in (a.d_k, a.d_v, a.d_sk, a.d_sv, a.d_mass)]
    a.mass = a.d_mass.cpu().numpy()
    a.k, a.v, a.sk, a.sv = (x.cpu().numpy() for x in start[:4])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.select()
        a.compact()
    for _ in range(3):
        for x, y in zip((a.d_k, a.d_v, a.d_sk, a.d_sv, a.d_mass), start):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        a.ok()
        a.check_select()
        a.check_compact(a.d_kept.cpu().numpy(), a.d_kept_lens.cpu().numpy())


CHILD = textwrap.dedent(r"""
    import os, sys
    sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]
    from test_gpu_evict import Cut, kev
    c = Cut(13, [3000, 2000], 700, 4, 30)
    c.select()
    kept, kept_lens = c.d_kept.cpu().numpy(), c.d_kept_lens.cpu().numpy()
    os.environ.update(KEV_TEST_STALL="1", KEV_TEST_WAIT_LIMIT="2000000")  # ~1 ms
    c.compact()
    assert kev.kev_read_status(c.status) == kev.binding.KEV_ERR_TIMEOUT
    del os.environ["KEV_TEST_STALL"], os.environ["KEV_TEST_WAIT_LIMIT"]
    c.kept, c.kept_lens = kept, kept_lens
    c.to_device()
    c.compact()
    c.ok()
    c.check_compact(kept, kept_lens)
    print("ALL OK")
""").replace("ROOT", repr(ROOT))


def test_a_wait_that_runs_out_is_reported():
    env = {k: v for k, v in os.environ.items() if k not in ("KEV_TEST_STALL", "KEV_TEST_WAIT_LIMIT")}
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0 and "ALL OK" in r.stdout, f"child failed:\n{r.stdout}\n{r.stderr[-4000:]}"
