"""GPU parity of kev_logprobs against its float64 definition.

Tolerances.  y = (x - max) log2e / T is off by a relative 2^-22 (three roundings), so e^y by a relative 2^-22 (1 + |y|)
(and 2^-22 for the exponential itself); only terms with |y| < 40 count.  A thread adds up at most V / 512 + 64 terms one
after the other, each addition off by 2^-24, and the joins add some 2^-24 each: with N = V / 512 + 64 the sum is off by a
relative (N + 256) 2^-24, and so is log S absolutely.  |log p| is off by that and 2^-21 |log p|.  The entropy is
log S - W / S, both parts not negative, W with the same relative error: (N + 256) 2^-23 (1 + H).
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

pytestmark = pytest.mark.gpu
INF = float("inf")


def run(x, dtype, tokens, temperature=None, top=0, active=None, **kw):
    n, v = x.shape
    x = torch.from_numpy(x.astype(np.float32)).to({"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]).cuda()
    lp, ent = torch.full((n,), 7.0, device="cuda"), torch.full((n,), 7.0, device="cuda")
    tt, tl = torch.full((n, max(top, 1)), -7, dtype=torch.int32, device="cuda"), torch.full((n, max(top, 1)), 7.0, device="cuda")
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    t = None if temperature is None else torch.tensor(temperature, dtype=torch.float32, device="cuda")
    a = None if active is None else torch.tensor(active, dtype=torch.uint8, device="cuda")
    tok = torch.tensor(tokens, dtype=torch.int32, device="cuda")
    kev.kev_logprobs(x, n, v, dtype, t, a, tok, lp, ent, top, tt if top else None, tl if top else None, status, **kw)
    st = kev.kev_read_status(status)
    return x.float().cpu().numpy(), st, lp.cpu().numpy(), ent.cpu().numpy(), tt.cpu().numpy(), tl.cpu().numpy()


def check(x, dtype, tokens, temperature=None, top=0):
    stored, st, lp, ent, tt, tl = run(x, dtype, tokens, temperature, top)
    assert st == 0
    t32 = None if temperature is None else np.asarray(temperature, np.float32)
    wlp, went, wtt, wtl = S.logprobs(stored, t32, tokens, top)
    n_add = (x.shape[1] / 512 + 64 + 256) * 2.0 ** -24

    def near(got, want, tol):
        fine = np.isfinite(want)
        np.testing.assert_array_equal(got[~fine], want[~fine].astype(np.float32))
        assert (np.abs(got[fine] - want[fine]) <= tol[fine]).all(), np.abs(got[fine] - want[fine]).max()

    with np.errstate(invalid="ignore"):
        near(lp, wlp, n_add + 2.0 ** -21 * np.abs(wlp))
        near(ent, went, 2 * n_add * (1 + np.abs(went)))
        if top:
            np.testing.assert_array_equal(tt, wtt)
            near(tl, wtl, n_add + 2.0 ** -21 * np.abs(wtl))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,v", [(1, 1), (3, 7), (2, 33), (5, 1000), (2, 4099), (1, 16384), (4, 32003), (3, 65537), (700, 257),
                                 (320, 33000), (1, 151936), (33, 151936)])
def test_rows(n, v, dtype):
    g = np.random.default_rng(n * v)
    x = 2.5 * g.standard_normal((n, v))
    check(x, dtype, g.integers(0, v, n), None, min(v, 20))
    check(x, dtype, x.argmax(-1), g.random(n) * 1.5 + 0.1, min(v, 1))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("top", [0, 1, 2, 5, 31, 32])
def test_tops_and_greedy_rows(top, dtype):
    g = np.random.default_rng(top)
    x = 2.5 * g.standard_normal((6, 30011))
    check(x, dtype, [int(np.argmax(x[0])), 5, int(np.argmax(x[2])), 0, 30010, 7], [0.0, 0.0, 1.0, 0.7, 0.0, 5.0], top)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 3, 400])
def test_orders_that_defeat_a_threshold(n, dtype):
    """Rows that are all equal, rise, fall, or hold their best tokens in the last places; many ties at every threshold."""
    v = 40000
    g = np.random.default_rng(1)
    up = np.arange(v) / v * 20 - 10
    rows = [np.zeros(v), up, up[::-1], -up ** 2, np.floor(up), np.floor(-up), np.where(np.arange(v) > v - 9, 3.0, -2.0),
            np.where(np.arange(v) % 977 == 3, 1.0, 0.5), -np.zeros(v), np.where(g.random(v) > 0.5, -0.0, 0.0)]
    x = np.stack([rows[i % len(rows)] for i in range(max(n, len(rows)))])
    check(x, dtype, [i * 37 % v for i in range(len(x))], None, 32)
    check(x, dtype, [i * 37 % v for i in range(len(x))], None, 3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v", [300, 20000, 70001])
def test_masked_rows(v, dtype):
    """A grammar's -infinity: over a run of tokens, almost everywhere, everywhere but one place; and rows left without a
    distribution."""
    g = np.random.default_rng(v)
    x = 2.5 * g.standard_normal((9, v))
    x[0, :v // 2] = -INF
    x[1, v // 3:] = -INF
    x[2, g.random(v) > 0.02] = -INF
    x[2, v // 2] = 0
    x[3] = -INF
    x[3, v - 1] = -4
    x[4] = -INF
    x[5, v // 7] = float("nan")
    x[6, v - 2] = INF
    x[7, :v - 40] = -INF
    x[8, :] = 1e38 if dtype == "fp32" else 1e30
    x[8, 0] = -1e38
    check(x, dtype, [v - 1, 0, v // 2, v - 1, 1, 2, 3, 0, 5], None, 25)
    check(x, dtype, [0, v - 1, v // 2, 0, 1, 2, 3, v - 1, 0], [1, 0, 2, 0, 0, 0, 1, 0.3, 1], 25)


def test_large_magnitudes_keep_their_differences():
    x = np.float32(1e6) + np.arange(64, dtype=np.float32).reshape(1, 64) / 8
    check(x, "fp32", [63], None, 5)
    check(x, "fp32", [0], [3.0], 5)


def test_tiny_temperatures():
    x = np.random.default_rng(3).standard_normal((3, 1000)).astype(np.float32)
    stored, st, lp, ent, tt, tl = run(x, "fp32", x.argmax(-1), [1e-30, 1e-40, 1e-8], 2)
    assert st == 0 and np.abs(lp).max() < 1e-6 and np.abs(ent).max() < 1e-6 and (tt[:, 0] == x.argmax(-1)).all() and (tl[:, 1] < -10).all()


def test_inactive_rows_are_left_as_they_are():
    x = np.random.default_rng(2).standard_normal((5, 500))
    x[1] = float("nan")
    stored, st, lp, ent, tt, tl = run(x, "bf16", [1, 10 ** 6, 2, -4, 3], [1.0, -1.0, 1.0, INF, 0.0], 4, active=[1, 0, 1, 0, 1])
    assert st == 0
    for r in (1, 3):
        assert lp[r] == 7 and ent[r] == 7 and (tt[r] == -7).all() and (tl[r] == 7).all()
    assert (lp[[0, 2]] < 0).all() and (tt[[0, 2, 4]] >= 0).all()


@pytest.mark.parametrize("n", [2, 900])
def test_device_errors_write_nothing(n):
    x = np.random.default_rng(2).standard_normal((n, 600))
    good = [1] * n
    for tokens, temperature in (([1] * (n - 1) + [600], None), ([-1] + [1] * (n - 1), None), (good, [1.0] * (n - 1) + [-0.5]),
                                (good, [float("nan")] + [1.0] * (n - 1)), (good, [1.0] * (n - 1) + [INF])):
        _, st, lp, ent, tt, tl = run(x, "bf16", tokens, temperature, 3)
        assert st == kev.binding.KEV_ERR_SAMPLING
        assert (lp == 7).all() and (ent == 7).all() and (tt == -7).all() and (tl == 7).all()


def test_outputs_not_wanted():
    x = torch.randn(4, 3001, device="cuda")
    ent = torch.zeros(4, device="cuda")
    kev.kev_logprobs(x, 4, 3001, "fp32", None, None, None, None, ent, 0, None, None, None)
    lp = torch.zeros(4, device="cuda")
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    kev.kev_logprobs(x, 4, 3001, "fp32", None, None, tok, lp, None, 0, None, None, None)
    want = torch.log_softmax(x.double(), -1)
    assert torch.allclose(lp.double(), want[:, 0], atol=1e-4)
    assert torch.allclose(ent.double(), -(want.exp() * want).sum(-1), atol=1e-4)


def test_captured_on_another_stream():
    n, v = 20, 50000
    x = torch.randn(n, v, device="cuda").bfloat16()
    tok = torch.arange(n, dtype=torch.int32, device="cuda")
    lp, ent, tt, tl = (torch.zeros(*s, device="cuda", dtype=d) for s, d in
                       (((n,), torch.float32), ((n,), torch.float32), ((n, 5), torch.int32), ((n, 5), torch.float32)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        kev.kev_logprobs(x, n, v, "bf16", None, None, tok, lp, ent, 5, tt, tl, status)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
    torch.cuda.synchronize()
    x.copy_(torch.randn(n, v, device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    want = torch.log_softmax(x.double(), -1)
    assert torch.allclose(lp.double(), want[torch.arange(n), tok.long()], atol=1e-4)
    assert (tl.double() - torch.topk(want, 5, -1)[0]).abs().max() < 1e-4


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHILD = textwrap.dedent(r"""
    import os, sys
    sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]
    import numpy as np
    from test_gpu_logprobs import check, kev, run
    for n, v in ((3, 151936), (700, 33000)):
        x = np.random.default_rng(n).standard_normal((n, v))
        os.environ.update(KEV_TEST_STALL="1", KEV_TEST_WAIT_LIMIT="2000000")  # ~1 ms
        assert run(x, "bf16", [1] * n, None, 5)[1] == kev.binding.KEV_ERR_TIMEOUT
        del os.environ["KEV_TEST_STALL"], os.environ["KEV_TEST_WAIT_LIMIT"]
        check(x, "bf16", [1] * n, None, 5)
    print("ALL OK")
""").replace("ROOT", repr(ROOT))


def test_a_wait_that_runs_out_is_reported():
    env = {k: v for k, v in os.environ.items() if k not in ("KEV_TEST_STALL", "KEV_TEST_WAIT_LIMIT")}
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0 and "ALL OK" in r.stdout, f"child failed:\n{r.stdout}\n{r.stderr[-4000:]}"
