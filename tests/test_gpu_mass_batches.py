"""kev_attn_mass_paged over batches of many questions, and on scores where its arithmetic shows.

Tolerances as derived in test_gpu_mass.py: a weight is off by a relative (8 (d + 8) + 8) S 2^-24, and the additions by n 2^-24
for n weights of a position.  With scores of a few hundredths what is left counts: the row's log sum is at most 9 for 500
positions, so it and the exponent of a weight are off by 2^-20 and 2^-21 (a last place, and half of one), ln 2 times that in
the weight; the exponential by 2^-22, in the weight and in the sum: 32 2^-24 altogether.  Weights rounded to fp16 (2^-11) or
bf16 (2^-8) would show."""
import numpy as np
import pytest
import torch

from oracle import serve_oracle as S

from test_gpu_mass import Mass

pytestmark = pytest.mark.gpu


def batch(n, longest):
    """Lengths with runs of empty questions at the beginning, in the middle and at the end, and prefixes of 0 to 3 pages."""
    g = np.random.default_rng(n)
    lens = np.where(g.random(n) < 0.3, 0, g.integers(1, longest + 1, n))
    for a, b in ((0, 0.1), (0.3, 0.45), (0.85, 1.0)):
        lens[int(a * n):int(b * n)] = 0
    prefix = g.integers(0, 100, n)
    prefix[g.random(n) < 0.05] = 300
    return lens.tolist(), prefix.tolist()


@pytest.mark.parametrize("n", [257, 600, 4096])
@pytest.mark.parametrize("longest,told", [(2, True), (2, False), (7, False)])
@pytest.mark.parametrize("dtype,pool", [("bf16", "bf16"), ("fp32", "fp32")])
def test_more_questions_than_threads(dtype, pool, longest, told, n):
    lens, prefix = batch(n, longest)
    m = Mass(40, lens, prefix, 4, 1, 64, dtype, pool)
    m.call(0.5, longest if told else 0)
    m.ok()
    m.check(0.5)


@pytest.mark.parametrize("dtype,pool", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32")])
@pytest.mark.parametrize("lens,prefix", [([0, 0, 0, 1], [0, 0, 0, 300]), ([1, 0, 0, 0], [200, 5, 5, 5]), ([0, 150, 0, 0, 2, 0], [1, 2, 3, 4, 500, 6])])
@pytest.mark.parametrize("told", [True, False])
def test_empty_questions_around(lens, prefix, told, dtype, pool):
    m = Mass(41, lens, prefix, 8, 2, 64, dtype, pool)
    m.call(1.0, max(lens) if told else 0)
    m.ok()
    m.check()


@pytest.mark.parametrize("factor", [0.0, 2.0 ** -8])
@pytest.mark.parametrize("lens,max_chunk", [([1, 1], 1), ([3, 1], 3), ([40, 7], 0)])
@pytest.mark.parametrize("dtype,pool,d", [("bf16", "bf16", 128), ("bf16", "e4m3", 128), ("fp32", "fp32", 64), ("fp32", "e4m3", 128)])
def test_small_scores_show_the_weights_rounding(dtype, pool, d, lens, max_chunk, factor):
    """Scores of zero, and of a few hundredths: every weight is near 1 / n, and right in the last places of fp32."""
    m = Mass(42, lens, [300, 77], 7, 1, d, dtype, pool)
    m.q *= factor
    m.call(0.0, max_chunk)
    m.ok()
    q = m.q.float().cpu().numpy().astype(np.float64)
    want, top = S.attn_mass(q, [k for k, _ in m.caches()], m.prefix, m.intervals, [m.positions(m.old, i) for i in range(2)], 0)
    rel = ((8 * (d + 8) + 8) * top + 32 + max(lens) * 7) * 2.0 ** -24
    assert rel < 2.0 ** -13
    got = m.mass.cpu().numpy()
    for i, y in enumerate(want):
        x = m.positions(got, i)
        assert (np.abs(x - y) <= rel * y).all(), (i, np.abs(x / y - 1).max(), rel)


@pytest.mark.parametrize("shift", [-124, -118, -110, -60, 60, 100])
@pytest.mark.parametrize("dtype,pool,d", [("bf16", "e4m3", 128), ("bf16", "e4m3", 64), ("bf16", "bf16", 128), ("fp32", "e4m3", 64)])
@pytest.mark.parametrize("lens,max_chunk", [([1, 1], 1), ([2, 1], 2), ([20, 40], 0)])
def test_small_q_and_large_k_and_the_other_way_round(lens, max_chunk, dtype, pool, d, shift):
    """Rows of q times 2^shift, cached K times 2^-shift: the scores are as without either."""
    m = Mass(43, lens, [300, 17], 8, 2, d, dtype, pool)
    m.q.copy_(torch.ldexp(m.q.double(), torch.tensor(shift, device="cuda")).to(m.q.dtype))
    pk, sk = m.pools[0]
    x = pk if sk is None else sk
    x.copy_(torch.ldexp(x.double(), torch.tensor(-shift, device="cuda")).to(x.dtype))
    m.call(1.0, max_chunk)
    m.ok()
    m.check()
