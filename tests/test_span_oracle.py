"""Pins of the oracle's span functions: closed forms, the plain prefill and decode, a library rounding, and planted mistakes."""
import numpy as np
import pytest
import torch

from oracle import kev_oracle as O


def test_e4m3_round_is_the_library_rounding_everywhere():
    """Every code, every midpoint between neighbours and its two fp32 neighbours, and random values."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    v = np.unique(codes[np.isfinite(codes)])
    mid = ((v[1:].astype(np.float64) + v[:-1]) / 2).astype(np.float32)
    rng = np.random.default_rng(0)
    x = np.concatenate([v, mid, np.nextafter(mid, np.float32(1e9)), np.nextafter(mid, np.float32(-1e9)),
                        (rng.standard_normal(20000) * np.exp(rng.uniform(-9, 5, 20000))).astype(np.float32)])
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(O.e4m3_round(x), want)
    assert O.e4m3_round(1e9) == 448 and O.e4m3_round(-460.0) == -448 and np.isnan(O.e4m3_round(np.nan))


def test_quantised_rows():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 128)).astype(np.float32) * np.exp(rng.uniform(-20, 20, (50, 1))).astype(np.float32)
    code, s = O.quantise_rows(x)
    back = code * s[:, None].astype(np.float64)
    # half an e4m3 step: relative 2^-4, or 2^-10 of the scale in the subnormal range, and the fp32 quotients
    assert (np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s[:, None]) * (1 + 1e-5)).all()
    top = np.abs(x).argmax(-1)
    np.testing.assert_array_equal(np.abs(code[np.arange(50), top]), 448.0)
    code, s = O.quantise_rows(np.zeros((2, 8), np.float32))
    assert (code == 0).all() and (s == 0).all()


@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 0), (3, 2), (1, 0), (40, 3)])
def test_visible_positions(window, sinks):
    for p in range(12):
        seen = O.span_visible(p, 12, window, sinks)
        for u in range(12):
            want = u <= p and (not window or u > p - window or u < sinks)
            assert seen[u] == want
        assert seen[p]  # every token sees itself: no row is empty


def test_without_a_window_it_is_the_prefill_and_in_chunks_too():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((9, 4, 16)), rng.standard_normal((9, 2, 16)), rng.standard_normal((9, 2, 16))
    iv = np.array([[0, 5], [6, 9]])
    ref = O.prefill(q, k, v, iv)
    out, size = O.span_attention(q, [k[0:5], k[6:9]], [v[0:5], v[6:9]], [0, 0], iv)
    np.testing.assert_allclose(out, ref, atol=1e-12)
    assert (size >= np.abs(out) - 1e-12).all()
    part, _ = O.span_attention(q[3:5], [k[0:5]], [v[0:5]], [3], [[0, 2]])
    np.testing.assert_allclose(part, ref[3:5], atol=1e-12)


def test_windows_against_an_explicit_mask_and_planted_mistakes():
    rng = np.random.default_rng(3)
    n, d = 14, 8
    q, k, v = (rng.standard_normal((n, 1, d)) for _ in range(3))

    def dense(vis):
        z = np.where(vis, q[:, 0] @ k[:, 0].T / np.sqrt(d), -np.inf)
        w = np.exp(z - z.max(-1, keepdims=True))
        return (w / w.sum(-1, keepdims=True)) @ v[:, 0]

    p, u = np.arange(n)[:, None], np.arange(n)[None, :]
    out, _ = O.span_attention(q, [k], [v], [0], [[0, n]], 4, 2)
    np.testing.assert_allclose(out[:, 0], dense((u <= p) & ((p - u < 4) | (u < 2))), atol=1e-12)
    for wrong in ((u <= p) & ((p - u <= 4) | (u < 2)), (u <= p) & (p - u < 4), (u <= p) & ((p - u < 4) | (u <= 2)),
                  (p - u < 4) | (u < 2)):
        assert np.abs(out[:, 0] - dense(wrong)).max() > 1e-3


def test_masked_positions_are_left_out():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((1, 2, 8)), rng.standard_normal((6, 1, 8)), rng.standard_normal((6, 1, 8))
    ref, _ = O.span_attention(q, [k], [v], [5], [[0, 1]], 2, 1)
    k[2], v[3] = np.inf, np.nan
    out, _ = O.span_attention(q, [k], [v], [5], [[0, 1]], 2, 1)
    np.testing.assert_array_equal(out, ref)


def test_validation():
    t = np.array([[0, 1, 2], [3, 4, 5]])
    iv = [[0, 3], [3, 5]]
    ok = dict(total_tokens=5, prefix_lens=[10, 200], table=t, n_blocks=6)
    assert O.validate_span(iv, **ok) is None
    assert O.validate_span([[0, 4], [3, 5]], **ok) == O.INTERVALS
    assert O.validate_span([[0, 3], [3, 6]], **ok) == O.INTERVALS
    assert O.validate_span(iv, **ok, max_chunk=2) == O.INTERVALS
    assert O.validate_span(iv, **{**ok, "prefix_lens": [-1, 0]}) == O.PREFIX
    assert O.validate_span(iv, **{**ok, "prefix_lens": [382, 0]}) == O.SLOT_OVERFLOW
    assert O.validate_span(iv, **{**ok, "n_blocks": 4}) == O.SLOT
    bad = t.copy()
    bad[1, 0] = 0
    assert O.validate_span(iv, **{**ok, "table": bad}) == O.SLOT
    assert O.validate_span(iv, **{**ok, "table": bad}, window=50) is None  # question 1's first page has left its window
    assert O.validate_span(iv, **{**ok, "table": bad}, window=50, sinks=1) == O.SLOT
    assert O.validate_span(iv, **{**ok, "table": bad}, attend=False) is None
