"""The bound on e4m3 rows that the C header states, down to rows whose scale is subnormal or zero."""
import numpy as np
import pytest

from oracle import kev_oracle as O


@pytest.mark.parametrize("exponent", [0, 60, 110, -100, -116, -118, -120, -125, -130, -135, -138, -140, -141, -142, -145, -149])
def test_quantised_rows_come_back_within_the_stated_bound(exponent):
    rng = np.random.default_rng(1000 + exponent)
    x = np.ldexp(rng.standard_normal((400, 64)), exponent).astype(np.float32)
    code, s = O.quantise_rows(x)
    back, x = code * s[:, None].astype(np.float64), x.astype(np.float64)
    place = np.where(s > 0, np.spacing(np.where(s > 0, s, 1)), 2.0 ** -149).astype(np.float64)[:, None]
    assert (np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s[:, None]) * (1 + 2.0 ** -20) + 224 * place).all()
    assert (code[s == 0] == 0).all()
