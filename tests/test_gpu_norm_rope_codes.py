"""kev_norm_rope_paged into an e4m3 cache: a key is quantised from its fp32 row, so its codes have one rounding behind them.

With y the definition's row, off by at most tol in fp32 (test_gpu_norm_rope.py: (d / 2 + 12) 2^-24 (|a| + |b|)), the scale is
max |y| / 448 to within tol / 448 and a rounding of 2^-24, and a code the e4m3 value nearest to some number within
tol / s + 2^-23 |y / s| of y / s.  Keys rounded to bf16 first (2^-8) would miss these codes in one of twenty places."""
import numpy as np
import pytest

from oracle import kev_oracle as O

from test_gpu_norm_rope import Norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,prefix", [([1, 5, 100], [200, 0, 60]), ([600, 30], [3, 127])])
@pytest.mark.parametrize("dtype,h_q,h_kv,d", [("bf16", 8, 2, 128), ("bf16", 4, 4, 64), ("fp32", 8, 2, 64)])
def test_the_codes_of_keys(dtype, h_q, h_kv, d, lens, prefix):
    n = Norm(20, lens, prefix, h_q, h_kv, d, dtype, "e4m3", start=[p + 9 for p in prefix])
    n.call(k_out=False)
    n.ok()
    (_, (k, tol)), _ = n.expect()
    pool, scale = n.pools[0]
    codes, scales = pool.float().cpu().numpy().astype(np.float64), scale.cpu().numpy().astype(np.float64)
    loose = 0
    for i, ((b, e), p) in enumerate(zip(n.intervals, prefix)):
        u = p + np.arange(e - b)
        at = (n.table[i, u // 128], slice(None), u % 128)
        y, t, c, s = k[b:e], tol[b:e], codes[at], scales[at]
        top = np.abs(y).max(-1)
        assert (np.abs(s * 448 - top) <= t.max(-1) + 2.0 ** -23 * top).all()
        x, off = y / s[..., None], t / s[..., None] + 2.0 ** -23 * np.abs(y / s[..., None])
        lo, hi = (O.e4m3_round(x + f) for f in (-off, off))
        assert ((lo <= c) & (c <= hi)).all()
        loose += int((lo != hi).sum())
    assert loose < 0.005 * k.size  # nearly every code is pinned
