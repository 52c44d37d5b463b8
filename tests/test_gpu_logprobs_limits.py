"""kev_logprobs where a wait gives up, and at the ends of what temperatures may be."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest

from test_gpu_logprobs import ROOT, check

pytestmark = pytest.mark.gpu

CHILD = textwrap.dedent(r"""
    import os, sys
    sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]
    import numpy as np
    from test_gpu_logprobs import S, kev, run
    for n, v in ((3, 151936), (20, 151936), (700, 33000)):
        x = np.random.default_rng(n).standard_normal((n, v))
        os.environ.update(KEV_TEST_STALL="1", KEV_TEST_WAIT_LIMIT="2000000")  # ~1 ms
        stored, st, lp, ent, tt, tl = run(x, "bf16", [1] * n, None, 5)
        del os.environ["KEV_TEST_STALL"], os.environ["KEV_TEST_WAIT_LIMIT"]
        assert st == kev.binding.KEV_ERR_TIMEOUT
        wlp, went, wtt, wtl = S.logprobs(stored, None, [1] * n, 5)
        left = (lp == 7) & (ent == 7) & (tt == -7).all(1) & (tl == 7).all(1)
        assert left[0], (n, lp[0], ent[0], tt[0], tl[0])
        for r in np.flatnonzero(~left):  # a row is left as it was, or whole and right
            assert abs(lp[r] - wlp[r]) < 1e-3 and abs(ent[r] - went[r]) < 1e-3 and (tt[r] == wtt[r]).all(), (n, r, tt[r], lp[r])
            assert np.abs(tl[r] - wtl[r]).max() < 1e-3
    print("ALL OK")
""").replace("ROOT", repr(ROOT))


def test_rows_whose_tiles_did_not_come_are_left_as_they_were():
    env = {k: v for k, v in os.environ.items() if k not in ("KEV_TEST_STALL", "KEV_TEST_WAIT_LIMIT")}
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0 and "ALL OK" in r.stdout, f"child failed:\n{r.stdout}\n{r.stderr[-4000:]}"


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [1e-28, 1e-31, 1e-34, 1e-37])
def test_tiny_temperatures_of_tiny_differences(size, dtype):
    """Logits of the temperature's size: the distribution is that of ordinary logits at temperature 1."""
    x = 2.5 * np.random.default_rng(5).standard_normal((3, 2000)) * size
    check(x, dtype, [int(x[0].argmax()), 7, 1999], [size, 2 * size, 0.5 * size], 4)
