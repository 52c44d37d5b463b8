"""The operators around the span attention over blocks whose elements lie past 2^32 from the pool's beginning: the same
results, bit for bit, as over the same blocks at its beginning."""
import numpy as np
import pytest
import torch

import packed_question_isolated_gb300 as kev

from test_gpu_evict import Cut
from test_gpu_mass import Mass
from test_gpu_norm_rope import Norm

pytestmark = pytest.mark.gpu
BLOCKS = 40000  # times 8 heads, 128 rows and 128 elements: 5.2e9 elements, 10.5 GB in bf16


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def far(x):
    """x's blocks as the last ones of a pool of zeros."""
    y = torch.zeros((BLOCKS,) + tuple(x.shape[1:]), dtype=torch.uint8 if x.element_size() == 1 else x.dtype, device="cuda")
    y[BLOCKS - x.shape[0]:] = x.view(y.dtype)
    return y.view(x.dtype)


def moved(s):
    first = BLOCKS - s.n_blocks
    s.pools = [(far(p), None if c is None else far(c)) for p, c in s.pools]
    s.table = np.where(s.table >= 0, s.table + first, -1).astype(np.int32)
    s.n_blocks = BLOCKS
    s.to_device()
    return first


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,max_chunk", [([1, 2], 2), ([40, 130], 0)])
def test_mass(lens, max_chunk, pool):
    a, b = (Mass(60, lens, [300, 1000], 16, 8, 128, "bf16", pool) for _ in range(2))
    first = moved(b)
    b.mass = far(b.mass)
    for m in (a, b):
        m.call(0.5, max_chunk)
        m.ok()
    a.check(0.5)
    assert (b.mass[first:] == a.mass).all() and (b.mass[:first] == 0).all()


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", [[5, 20], [500, 200]])
def test_norm_rope(lens, pool):
    a, b = (Norm(61, lens, [300, 1000], 16, 8, 128, "bf16", pool) for _ in range(2))
    first = moved(b)
    for n in (a, b):
        n.call()
        n.ok()
    assert (a.q_out == b.q_out).all()
    for x, y in ((x, y) for p, q in zip(a.pools, b.pools) for x, y in zip(p, q) if x is not None):
        assert (x.view(torch.uint8) == y[first:].view(torch.uint8)).all()
        assert not y[:first:997].view(torch.uint8).any()


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_select_and_compact(pool):
    c = Cut(62, [3000, 700, 100], 400, 4, 30, h_kv=8, d=128, pool=pool)
    first = BLOCKS - c.n_blocks
    k, v, sk, sv, mass = (far(x) for x in (c.d_k, c.d_v, c.d_sk, c.d_sv, c.d_mass))
    table = torch.where(c.d_table >= 0, c.d_table + first, c.d_table)
    c.select()
    c.ok()
    c.check_select()
    kept = c.d_kept.clone()
    c.compact()
    c.ok()
    c.check_compact(kept.cpu().numpy(), c.d_kept_lens.cpu().numpy())
    c.d_kept.fill_(-9)
    e4m3 = pool == "e4m3"
    cache = kev.make_paged_cache(k, v, table, c.width, BLOCKS, pool, sk if e4m3 else None, sv if e4m3 else None)
    kev.kev_select_paged(mass, c.d_lens, None, 3, table, c.width, BLOCKS, c.keep, 4, 30, c.d_kept, c.d_kept_lens, *c.end())
    kev.kev_compact_paged(c.d_kept, c.keep, c.d_lens, c.d_kept_lens, 3, cache, mass, *c.end())
    c.ok()
    assert (c.d_kept == kept).all()
    for i, m in enumerate(c.d_kept_lens.tolist()):
        u = np.arange(m)
        block, row = torch.from_numpy(c.table[i, u // 128].astype(np.int64)).cuda(), torch.from_numpy(u % 128).cuda()
        for x, y in ((k, c.d_k), (v, c.d_v), (mass, c.d_mass)) + (((sk, c.d_sk), (sv, c.d_sv)) if e4m3 else ()):
            assert (x[block + first, :, row] == y[block, :, row]).all()


def test_logprobs():
    n, v = 2200, 2 ** 21 + 1  # the last rows lie past 2^32 elements
    x = torch.zeros(n, v, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(63)
    rows = torch.tensor([0, 1023, 1024, 2047, 2048, n - 1], device="cuda")
    for r in rows.tolist():
        x[r] = torch.randn(v, generator=g, device="cuda").bfloat16()
    tok = (torch.arange(n, device="cuda") * 911).int()

    def call(x, tok):
        m = len(x)
        lp, ent, tl = torch.zeros(m, device="cuda"), torch.zeros(m, device="cuda"), torch.zeros(m, 5, device="cuda")
        tt, st = torch.zeros(m, 5, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        kev.kev_logprobs(x, m, v, "bf16", None, None, tok, lp, ent, 5, tt, tl, st)
        assert kev.kev_read_status(st) == 0
        return lp, ent, tt, tl

    got = call(x, tok)
    for r in rows.tolist():  # the same rows alone: of parts of a cluster, so sums may differ in the last places
        lp, ent, tt, tl = call(x[r:r + 1].clone(), tok[r:r + 1].clone())
        assert (got[2][r] == tt[0]).all() and (got[3][r] - tl[0]).abs().max() < 1e-4
        assert abs(got[0][r] - lp[0]) < 1e-4 and abs(got[1][r] - ent[0]) < 1e-4
