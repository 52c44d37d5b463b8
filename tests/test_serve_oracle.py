"""The float64 definitions of the operators around the span attention, on cases worked out by hand (no GPU)."""
import numpy as np

from oracle import serve_oracle as S


def test_norm_rope_by_hand():
    x = np.zeros((2, 1, 4))
    x[:, 0] = [3.0, 0.0, 4.0, 0.0]  # mean square 25/4
    got = S.norm_rope(x, np.array([1.0, 1.0, 2.0, 1.0]), 0.0, [0, 1], 1e4)
    np.testing.assert_allclose(got[0, 0], [1.2, 0, 3.2, 0], atol=1e-12)  # position 0: no turn
    np.testing.assert_allclose(got[1, 0], [1.2 * np.cos(1) - 3.2 * np.sin(1), 0, 3.2 * np.cos(1) + 1.2 * np.sin(1), 0],
                               atol=1e-12)
    assert (S.norm_rope(x, None, 1.0, [0, 0], 1e4) == x).all()


def test_mass_by_hand():
    # one q-head, equal scores: token 0 at position 1 spreads 1 over 2 positions, token 1 over 3
    q, k = np.zeros((2, 1, 4)), np.zeros((3, 1, 4))
    new, _ = S.attn_mass(q, [k], [1], [(0, 2)], [np.full((3, 1), 10.0)], 0.5)
    np.testing.assert_allclose(new[0][:, 0], [5 + 1 / 2 + 1 / 3, 1 / 2 + 1 / 3, 1 / 3])
    fresh, _ = S.attn_mass(q, [k], [1], [(0, 2)], [np.full((3, 1), np.nan)], 0)
    np.testing.assert_allclose(fresh[0].sum(), 2)  # every token hands out 1


def test_select_by_hand():
    m = np.array([[0.0], [5], [1], [5], [2], [0]])
    assert S.select(m, 4, 1, 1).tolist() == [[0, 1, 3, 5]]
    assert S.select(m, 3, 1, 1).tolist() == [[0, 1, 5]]  # a tie: the lower position
    assert S.select(m, 6, 1, 1).tolist() == [list(range(6))]
    m[4] = np.nan
    assert S.select(m, 2, 0, 0).tolist() == [[1, 4]]


def test_logprobs_by_hand():
    x = np.log(np.array([[1.0, 2, 1, 4], [1, 1, 1, 1]]))
    lp, ent, top, top_lp = S.logprobs(x, None, [1, 2], 3)
    np.testing.assert_allclose(lp, np.log([0.25, 0.25]))
    np.testing.assert_allclose(ent, [1.75 * np.log(2), np.log(4)])
    assert top.tolist() == [[3, 1, 0], [0, 1, 2]]
    np.testing.assert_allclose(np.exp(top_lp[0]), [0.5, 0.25, 0.125])
    lp, ent, _, top_lp = S.logprobs(x, [0, 0], [3, 2], 2)
    assert lp.tolist() == [0, -np.inf] and ent.tolist() == [0, 0] and top_lp[0].tolist() == [0, -np.inf]
    assert np.isnan(S.logprobs(np.full((1, 3), -np.inf), None, [0], 1)[0][0])
