"""Lists longer than positions go are refused on the host (nothing is launched; addresses are never read on the host)."""
import pytest

from test_evict_abi import compact, lib, select  # noqa: F401


@pytest.mark.parametrize("keep", [2 ** 30 + 1, 2 ** 31 - 2048, 2 ** 31 - 64, 2 ** 31 - 1])
@pytest.mark.parametrize("n", [1, 2])
def test_keep_past_the_last_position(lib, n, keep):  # noqa: F811
    kw = dict(n=n, keep=keep, shape=lib.make_shape(1, 1, 128, "bf16"))
    assert select(lib, **kw) == lib.binding.KEV_ERR_UNSUPPORTED
    assert compact(lib, **kw) == lib.binding.KEV_ERR_UNSUPPORTED
    assert lib.kev_evict_workspace_size(n, keep, kw["shape"]) == 0


def test_the_longest_list_has_a_workspace(lib):  # noqa: F811
    chunks = 2 ** 30 // 64
    assert lib.kev_evict_workspace_size(1, 2 ** 30, lib.make_shape(1, 1, 128, "bf16")) >= 4 * chunks
    assert lib.kev_evict_workspace_size(8, 2 ** 30, lib.make_shape(8, 8, 128, "bf16")) >= 4 * 64 * chunks
    assert lib.kev_evict_workspace_size(8, 2 ** 30, lib.make_shape(16, 16, 128, "bf16")) == 0


@pytest.mark.parametrize("n,keep,h_kv", [(4096, 2 ** 30, 2 ** 30), (4096, 64, 2 ** 31 - 1), (1, 2 ** 30, 2 ** 25)])
def test_no_size_wraps(lib, n, keep, h_kv):  # noqa: F811
    assert lib.kev_evict_workspace_size(n, keep, lib.make_shape(h_kv, h_kv, 128, "bf16")) == 0


def test_shapes_that_a_move_does_not_take(lib):  # noqa: F811
    for shape, code in ((lib.make_shape(8, 2, 96, "bf16"), "UNSUPPORTED"), (lib.make_shape(7, 2, 128, "bf16"), "UNSUPPORTED"),
                        (lib.make_shape(8, 2, 128, 2), "UNSUPPORTED"), (lib.make_shape(8, 2, 128, "bf16", -1.0), "INVALID_ARG"),
                        (lib.make_shape(8, 0, 128, "bf16"), "INVALID_ARG")):
        assert compact(lib, shape=shape) == getattr(lib.binding, "KEV_ERR_" + code)
    for h_kv in (0, -2):
        assert select(lib, shape=lib.make_shape(8, h_kv, 128, "bf16")) == lib.binding.KEV_ERR_INVALID_ARG
        assert lib.kev_evict_workspace_size(2, 8, lib.make_shape(8, h_kv, 128, "bf16")) == 0
    assert lib.kev_evict_workspace_size(3, 64, lib.make_shape(0, 2, 96, 2, -1.0)) == lib.kev_evict_workspace_size(3, 64, lib.make_shape(8, 2, 128, "bf16"))
