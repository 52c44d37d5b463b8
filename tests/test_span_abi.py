"""Host-side refusals and workspace sizes of the span operators, without a GPU (nothing is launched)."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from packed_question_isolated_gb300 import build
    build.build()
    import packed_question_isolated_gb300 as kev
    return kev


def _span_args(lib, **kw):
    """Arguments of a valid-looking kev_chunk_attn_paged call (addresses are never read on the host)."""
    c = dict(q=0x1000, k=0x1000, v=0x1000, T=8, iv=0x1000, n=2, pre=0x1000, max_chunk=0, window=0, sinks=0, out=0x1000,
             shape=lib.make_shape(8, 2, 128, "bf16"), ws=0x1000, status=None, pool="bf16", pool_k=0x1000, pool_v=0x1000,
             table=0x1000, max_blocks=4, n_blocks=64, ks=None, vs=None)
    c.update(kw)
    c["bytes"] = kw.get("bytes", 1 << 40)
    c["cache"] = lib.make_paged_cache(c["pool_k"], c["pool_v"], c["table"], c["max_blocks"], c["n_blocks"], c["pool"],
                                      c["ks"], c["vs"])
    return c


REFUSED = [
    (dict(q=None), "INVALID_ARG"), (dict(k=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"),
    (dict(q=0x1008), "INVALID_ARG"), (dict(k=0x1004), "INVALID_ARG"), (dict(out=0x1002), "INVALID_ARG"),
    (dict(T=-1), "INVALID_ARG"), (dict(n=-1), "INVALID_ARG"), (dict(iv=None), "INVALID_ARG"), (dict(iv=0x1004), "INVALID_ARG"),
    (dict(pre=None), "INVALID_ARG"), (dict(pre=0x1002), "INVALID_ARG"), (dict(window=-1), "INVALID_ARG"),
    (dict(sinks=-1), "INVALID_ARG"), (dict(max_chunk=-1), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"),
    (dict(ws=0x1080), "INVALID_ARG"), (dict(bytes=64), "INVALID_ARG"), (dict(status=0x1002), "INVALID_ARG"),
    (dict(pool_k=None), "INVALID_ARG"), (dict(pool_v=0x1008), "INVALID_ARG"), (dict(table=None), "INVALID_ARG"),
    (dict(table=0x1002), "INVALID_ARG"), (dict(max_blocks=0), "INVALID_ARG"), (dict(n_blocks=0), "INVALID_ARG"),
    (dict(pool="e4m3"), "INVALID_ARG"), (dict(pool="e4m3", ks=0x1000, vs=0x1004), "INVALID_ARG"),
    (dict(pool="fp32"), "UNSUPPORTED"), (dict(n=4097), "UNSUPPORTED"), (dict(n_blocks=(1 << 20) + 1), "UNSUPPORTED"),
    (dict(max_blocks=(1 << 23) + 1), "UNSUPPORTED"), (dict(pool=7), "UNSUPPORTED"),
]


@pytest.mark.parametrize("kw,code", REFUSED)
def test_span_calls_refuse_on_the_host(lib, kw, code):
    want = getattr(lib.binding, "KEV_ERR_" + code)
    c = _span_args(lib, **kw)
    end = (c["shape"], c["ws"], c["bytes"], c["status"], 0)
    got = lib.kev_chunk_attn_paged(c["q"], c["k"], c["v"], c["T"], c["iv"], c["n"], c["pre"], c["max_chunk"], c["cache"],
                                   c["window"], c["sinks"], c["out"], *end, check=False)
    assert got == want
    if not {"q", "out", "window", "sinks", "max_chunk"} & set(kw):
        for f in (lib.kev_paged_write, lib.kev_paged_read):
            assert f(c["k"], c["v"], c["T"], c["iv"], c["n"], c["pre"], c["cache"], *end, check=False) == want
    if {"q", "k", "v", "out", "T", "n", "iv", "window", "sinks", "ws", "bytes", "status"} & set(kw) and kw != dict(n=4097):
        assert lib.kev_prefill_attn_window(c["q"], c["k"], c["v"], c["T"], c["iv"], c["n"], c["window"], c["sinks"], c["out"],
                                           *end, check=False) == want


@pytest.mark.parametrize("q,k,v,out", [  # 8 tokens: 16,384 bytes of q and out, 4,096 of k and v
    (0x100000, 0x200000, 0x300000, 0x100000), (0x100000, 0x200000, 0x300000, 0x103ff0),
    (0x103ff0, 0x200000, 0x300000, 0x100000), (0x100000, 0x200ff0, 0x300000, 0x201fe0), (0x100000, 0x200000, 0x303ff0, 0x300000)])
def test_out_over_an_input_is_refused(lib, q, k, v, out):
    c = _span_args(lib)
    end = (c["shape"], c["ws"], c["bytes"], None, 0)
    assert lib.kev_chunk_attn_paged(q, k, v, 8, c["iv"], 2, c["pre"], 0, c["cache"], 0, 0, out, *end,
                                    check=False) == lib.binding.KEV_ERR_INVALID_ARG
    assert lib.kev_prefill_attn_window(q, k, v, 8, c["iv"], 2, 0, 0, out, *end, check=False) == lib.binding.KEV_ERR_INVALID_ARG


@pytest.mark.parametrize("shape,code", [((8, 3, 128, "bf16"), "UNSUPPORTED"), ((34, 2, 128, "bf16"), "UNSUPPORTED"),
                                        ((8, 2, 96, "fp32"), "UNSUPPORTED"), ((8, 2, 256, "fp32"), "UNSUPPORTED"),
                                        ((8, 2, 128, "e4m3"), "UNSUPPORTED"), ((0, 2, 128, "bf16"), "INVALID_ARG"),
                                        ((8, 2, 128, "bf16", float("nan")), "INVALID_ARG")])
def test_span_shapes_refused(lib, shape, code):
    s = lib.make_shape(*shape[:3], {"bf16": 0, "fp32": 1, "e4m3": 2}[shape[3]], *shape[4:])
    c = _span_args(lib, shape=s)
    want = getattr(lib.binding, "KEV_ERR_" + code)
    assert lib.kev_paged_workspace_size(2, 8, s) == 0
    assert lib.kev_chunk_attn_paged(c["q"], c["k"], c["v"], 8, c["iv"], 2, c["pre"], 0, c["cache"], 0, 0, c["out"], s, c["ws"],
                                    c["bytes"], None, 0, check=False) == want


def test_span_workspace_sizes(lib):
    s = lib.make_shape(8, 2, 128, "bf16")
    sizes = [lib.kev_paged_workspace_size(4, t, s) for t in (0, 1, 4, 64, 1000, 2 ** 31 - 1)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert sizes[-1] >= 24 * (2 ** 31 // 4)  # 64-bit arithmetic
    assert lib.kev_paged_workspace_size(4097, 4, s) == 0 and lib.kev_paged_workspace_size(-1, 4, s) == 0
