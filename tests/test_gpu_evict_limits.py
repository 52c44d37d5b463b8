"""The move of kept rows when its waits run out; the shape that a selection takes."""
import os
import subprocess
import sys
import textwrap

import pytest

from test_gpu_evict import ROOT, Cut, kev

pytestmark = pytest.mark.gpu

CHILD = textwrap.dedent(r"""
    import os, sys
    sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]
    import numpy as np
    from test_gpu_evict import Cut, kev
    for pool in ("bf16", "e4m3"):
        c = Cut(13, [3000, 2000, 50], 700, 4, 30, pool=pool)
        c.select()
        kept, kept_lens = c.d_kept.cpu().numpy(), c.d_kept_lens.cpu().numpy()
        os.environ.update(KEV_TEST_STALL="1", KEV_TEST_WAIT_LIMIT="2000000")  # ~1 ms
        c.compact()
        assert kev.kev_read_status(c.status) == kev.binding.KEV_ERR_TIMEOUT
        del os.environ["KEV_TEST_STALL"], os.environ["KEV_TEST_WAIT_LIMIT"]
        # the first chunk of every list says nothing, so those behind it waited until the call gave up, and moved nothing
        for before, after, moved in zip((c.k, c.v, c.sk, c.sv, c.mass), c.state(), (1, 1, pool == "e4m3", pool == "e4m3", 1)):
            for i in (0, 1):
                x, y = c.rows(before, i, c.lens[i]), c.rows(after, i, c.lens[i])
                assert (x[64:] == y[64:]).all(), i
                for g in range(c.h_kv):
                    assert (y[:64, g] == (x[kept[i, g, :64], g] if moved else x[:64, g])).all(), (i, g)
            assert (c.rows(before, 2, 50) == c.rows(after, 2, 50)).all()
        c.kept, c.kept_lens = kept, kept_lens
        c.to_device()
        c.compact()
        c.ok()
        c.check_compact(kept, kept_lens)
    print("ALL OK")
""").replace("ROOT", repr(ROOT))


def test_the_wait_for_lower_chunks_gives_up():
    env = {k: v for k, v in os.environ.items() if k not in ("KEV_TEST_STALL", "KEV_TEST_WAIT_LIMIT")}
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0 and "ALL OK" in r.stdout, f"child failed:\n{r.stdout}\n{r.stderr[-4000:]}"


@pytest.mark.parametrize("h_q,d,dtype,scale", [(0, 0, "bf16", 0.0), (7, 96, 2, -1.0), (64, 128, "fp32", float("nan"))])
def test_of_a_selections_shape_only_the_kv_heads_count(h_q, d, dtype, scale):
    c = Cut(14, [500, 100, 300], 64, 2, 10)
    c.shape = kev.make_shape(h_q, c.h_kv, d, dtype, scale)
    assert kev.kev_evict_workspace_size(3, 64, c.shape) == c.bytes
    c.select()
    c.ok()
    c.check_select()
