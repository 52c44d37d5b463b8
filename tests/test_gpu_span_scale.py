"""The span operators with a scale of the caller's, which every kernel folds in at a place of its own, and decode over e4m3
held to the precision of its fp16 weights.  Tolerances as derived in test_gpu_span_values.py."""
import numpy as np
import pytest
import torch

from test_gpu_span import Span
from test_gpu_span_values import against_oracle, with_scale

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32"), ("fp32", "e4m3")]
SCALES = [1.0, 0.3, 0.02, 2.0 ** -40]


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("mask", [(0, 0), (100, 4)])
@pytest.mark.parametrize("dtype,pool", TYPES)
def test_chunks_with_a_scale(dtype, pool, mask, scale):
    b = with_scale(Span(500, [3, 0, 70, 1], [5, 9, 250, 600], 8, 2, 128, dtype, pool, gaps=1), scale)
    b.chunk(*mask)
    b.ok()
    against_oracle(b, b.caches(), mask, scale)


@pytest.mark.parametrize("scale", [None] + SCALES)
@pytest.mark.parametrize("mask", [(0, 0), (200, 4)])
@pytest.mark.parametrize("h_q,h_kv,d", [(8, 2, 128), (16, 1, 128), (6, 6, 64), (12, 1, 64)])
@pytest.mark.parametrize("dtype,pool", TYPES)
def test_decode_with_a_scale(dtype, pool, h_q, h_kv, d, mask, scale):
    b = with_scale(Span(501 + d, [1, 1, 0, 1, 1, 1], [0, 128, 50, 511, 2500, 640], h_q, h_kv, d, dtype, pool), scale)
    b.chunk(*mask, max_chunk=1)
    b.ok()
    against_oracle(b, b.caches(), mask, scale, weights=2.0 ** -11 if (dtype, pool) == ("bf16", "e4m3") else 2.0 ** -8)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_mixed_rounds_with_a_scale(pool, scale):
    r = np.random.default_rng(502)
    lens = [1] * 30 + [60, 2, 0, 40, 3]
    prefix = r.integers(0, 400, len(lens)).tolist()
    b = with_scale(Span(502, lens, prefix, 8, 2, 128, "bf16", pool, order=r.permutation(len(lens)).tolist()), scale)
    b.chunk()
    b.ok()
    against_oracle(b, b.caches(), scale=scale)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("h_q,h_kv,d", [(8, 2, 128), (7, 1, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_packed_windows_with_a_scale(dtype, h_q, h_kv, d, scale):
    lens = [1, 90, 0, 150]
    b = with_scale(Span(503, lens, [0] * 4, h_q, h_kv, d, dtype, order=[3, 1, 0, 2]), scale)
    b.packed(60, 3)
    b.ok()
    k, v = (x.float().cpu().numpy().astype(np.float64) for x in (b.k, b.v))
    against_oracle(b, [(k[s:e], v[s:e]) for s, e in b.intervals], (60, 3), scale)


@pytest.mark.parametrize("h_q,h_kv,d,mask", [(8, 2, 128, (0, 0)), (16, 1, 64, (300, 2)), (4, 4, 64, (0, 0))])
def test_decode_over_e4m3_with_weights_that_span_a_wide_range(h_q, h_kv, d, mask):
    """Peaked and flat rows, V rows of sizes from 2^-30 to 2^30: the weights of fp16 with a unit of their own."""
    b = Span(504, [1] * 6, [900, 130, 40, 2000, 0, 511], h_q, h_kv, d, "bf16", "e4m3")
    g = torch.Generator(device="cuda").manual_seed(504)
    b.q *= torch.exp2(torch.randint(-4, 4, (b.T, h_q, 1), generator=g, device="cuda").float()).to(b.q.dtype)
    b.write()
    sv = b.pools[1][1]
    sv *= torch.exp2(torch.randint(-30, 31, sv.shape, generator=g, device="cuda").float())
    b.chunk(*mask, max_chunk=1, write=False)
    b.ok()
    against_oracle(b, b.caches(), mask, weights=2.0 ** -11)
