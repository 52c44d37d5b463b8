"""The span operators at their limits: caches past 2^31 elements, many questions, windows as large as an int, the
timeout path of their kernels, and launch counts."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

import packed_question_isolated_gb300 as kev
from oracle import kev_oracle as O

from test_gpu_span import PAGE, Span, _kv

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("pool,lens,mc", [("bf16", [1, 1], 1), ("e4m3", [1, 1], 1), ("bf16", [70, 40], 0), ("e4m3", [70, 40], 0)])
def test_blocks_past_2_to_the_31_elements(pool, lens, mc):
    """The last blocks of a pool of 2.3e9 elements: element offsets past 32 bits, row coordinates near 2^31."""
    b = Span(200, lens, [200, 100], 8, 8, 128, "bf16", pool)
    n = 17800  # blocks of 8 x 128 x 128 elements
    dt = torch.bfloat16 if pool == "bf16" else torch.float8_e4m3fn
    pools = []
    for p, s in b.pools:
        big = torch.empty((n, 8, PAGE, 128), dtype=dt, device="cuda")
        big[n - b.n_blocks:].view(torch.uint8).copy_(p.view(torch.uint8))
        sc = None
        if s is not None:
            sc = torch.empty((n, 8, PAGE), device="cuda")
            sc[n - b.n_blocks:] = s
        pools.append((big, sc))
    assert pools[0][0].numel() > 2 ** 31
    small, b.pools = b.pools, pools
    shift, b.n_blocks = n - b.n_blocks, n
    b.table = np.where(b.table >= 0, b.table + shift, b.table)
    b.to_device()
    b.chunk(max_chunk=mc)
    b.ok()
    b.pools = [(p[shift:], None if s is None else s[shift:]) for p, s in pools]
    b.table = np.where(b.table >= 0, b.table - shift, b.table)
    b.check(*_kv(b.caches()), 0, 0)


@pytest.mark.parametrize("n", [1024, 4096])
def test_many_questions_sorted_and_not(n):
    r = np.random.default_rng(n)
    for order in (None, r.permutation(n).tolist()):
        b = Span(n, [1] * n, r.integers(0, 20, n).tolist(), 2, 1, 64, "bf16", "e4m3", order=order)
        b.chunk(max_chunk=1)
        b.ok()
        b.check(*_kv(b.caches()), 0, 0)


@pytest.mark.parametrize("mask", [(2 ** 31 - 1, 0), (2 ** 30, 2 ** 31 - 1), (1, 2 ** 31 - 1), (2 ** 30 + 5, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_windows_and_sinks_as_large_as_an_int(dtype, mask):
    b = Span(201, [30, 1, 140], [300, 129, 5], 8, 2, 64, dtype, dtype)
    b.chunk(*mask)
    b.ok()
    b.check(*_kv(b.caches()), 0, 0)  # everything is seen
    b.prefix = [0, 0, 0]
    b.packed(*mask)
    b.ok()
    k, v = (x.float().cpu().numpy().astype(np.float64) for x in (b.k, b.v))
    b.check([k[s:e] for s, e in b.intervals], [v[s:e] for s, e in b.intervals], 0, 0)


def test_group_of_sixteen_and_several_tokens_per_question():
    """max_chunk * G up to 16 rows: two 8-row tiles of the kernel for few rows, tokens across a page's end."""
    for h_q, h_kv, lens, prefix in ((16, 1, [1, 1, 0, 1], [127, 500, 3, 0]), (8, 2, [4, 3, 2, 1], [126, 254, 0, 700]),
                                    (5, 5, [16, 1, 9, 8], [120, 0, 127, 640]), (6, 2, [5, 2, 1, 4], [1, 255, 130, 900])):
        for pool in ("bf16", "e4m3"):
            for d in (64, 128):
                for mask in ((0, 0), (6, 1)):
                    b = Span(202, lens, prefix, h_q, h_kv, d, "bf16", pool)
                    b.chunk(*mask, max_chunk=max(lens))
                    b.ok()
                    b.check(*_kv(b.caches()), *mask)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_values_whose_sizes_differ_by_millions(pool):
    """One cached row is 2^20 times the others: with little weight it must not cost the others their precision."""
    for lens, mc in (([1, 1], 1), ([40, 30], 0)):
        b = Span(203, lens, [300, 150], 4, 2, 128, "bf16", pool)
        b.write()
        pv, sv = b.pools[1]
        for i in range(2):
            blk = int(b.table[i, 0])
            if sv is None:
                pv[blk, :, 60] *= 2.0 ** 20
            else:
                sv[blk, :, 60] *= 2.0 ** 20
            kp, ks = b.pools[0]
            if ks is None:
                kp[blk, :, 60] = 0
            else:
                kp.view(torch.uint8)[blk, :, 60] = 0
        b.chunk(max_chunk=mc, write=False)
        b.ok()
        b.check(*_kv(b.caches()), 0, 0)


def test_launch_counts():
    b = Span(204, [1, 1], [5, 9], 8, 2, 64)
    assert kev.kev_launch_count(19) == 3
    b.write()
    kev.kev_paged_read(b.k, b.v, b.T, b.iv, 2, b.pre, b.cache, *b.end())
    assert kev.kev_launch_count(16) == 1 and kev.kev_launch_count(17) == 1
    b.chunk(max_chunk=1)
    assert kev.kev_launch_count(18) == 2
    b = Span(205, [90, 1], [5, 9], 8, 2, 64)
    b.chunk()
    assert kev.kev_launch_count(18) == 4
    c = Span(206, [513], [5], 8, 2, 64)
    c.write()
    kev.kev_paged_read(c.k, c.v, c.T, c.iv, 1, c.pre, c.cache, *c.end())
    assert kev.kev_launch_count(16) == 2 and kev.kev_launch_count(17) == 2
    c.ok()
    b.chunk(write=False)
    assert kev.kev_launch_count(18) == 3
    b.ok()


CHILD = textwrap.dedent(r"""
    import os, sys
    sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]
    import packed_question_isolated_gb300 as kev
    from test_gpu_span import Span, _kv
    for pool in ("bf16", "e4m3"):
        for lens, mc in (([1, 1, 1], 1), ([300, 1, 40], 0)):
            b = Span(300, lens, [700, 130, 5], 8, 2, 128, "bf16", pool)
            os.environ["KEV_TEST_STALL"], os.environ["KEV_TEST_WAIT_LIMIT"] = "1", "2000000"  # about 1 ms
            assert b.chunk(max_chunk=mc) == 0
            assert kev.kev_read_status(b.status) == kev.binding.KEV_ERR_TIMEOUT
            os.environ.pop("KEV_TEST_STALL"), os.environ.pop("KEV_TEST_WAIT_LIMIT")
            b.chunk(max_chunk=mc)  # the same workspace, as the failed call left it
            b.ok()
            b.check(*_kv(b.caches()), 0, 0)
    print("ALL OK")
""").replace("ROOT", repr(ROOT))


def test_timeouts_are_reported_and_the_next_call_is_correct():
    """CTA 0 of the attention kernels first waits on a barrier that nothing arrives on, with a short limit: the call
    reports KEV_ERR_TIMEOUT and returns, and the next one on the same workspace is right."""
    env = {k: v for k, v in os.environ.items() if k not in ("KEV_TEST_STALL", "KEV_TEST_WAIT_LIMIT")}
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and "ALL OK" in r.stdout, f"{r.stdout}\n{r.stderr[-4000:]}"
