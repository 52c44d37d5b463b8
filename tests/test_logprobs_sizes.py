"""Row counts that 32-bit row numbers would wrap at are refused on the host (nothing is launched)."""
import pytest

from test_evict_abi import lib, logprobs  # noqa: F401


@pytest.mark.parametrize("n", [2 ** 30 + 1, 2 ** 31 - 512, 2 ** 31 - 1])
def test_too_many_rows(lib, n):  # noqa: F811
    for vocab in (1, 3):
        assert logprobs(lib, n=n, vocab=vocab, top=0) == lib.binding.KEV_ERR_UNSUPPORTED
