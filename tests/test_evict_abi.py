"""Host-side refusals and workspace sizes of the operators around the span attention, without a GPU (nothing is launched;
addresses are never read on the host)."""
import pytest

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    from packed_question_isolated_gb300 import build
    build.build()
    import packed_question_isolated_gb300 as kev
    return kev


def _cache(lib, c):
    if c["no_cache"]:
        return None
    return lib.make_paged_cache(c["pool_k"], c["pool_v"], c["table"], c["max_blocks"], c["n_blocks"], c["pool"], c["ks"], c["vs"])


def _defaults(lib, kw):
    c = dict(T=8, iv=0x1000, n=2, pre=0x1000, shape=lib.make_shape(8, 2, 128, "bf16"), ws=0x1000, bytes=1 << 40, status=None,
             pool="bf16", pool_k=0x1000, pool_v=0x1000, table=0x1000, max_blocks=4, n_blocks=64, ks=None, vs=None, no_cache=False)
    c.update(kw)
    return c


def norm_rope(lib, **kw):
    c = dict(q=0x100000, k=0x200000, v=0x300000, qs=0, ks_=0, vs_=0, q_out=0x400000, k_out=0x500000, pos=None, qw=None, kw=None,
             eps=1e-6, rope=0x1000, max_pos=64)
    c.update(_defaults(lib, {}))
    c.update(kw)
    return lib.kev_norm_rope_paged(c["q"], c["k"], c["v"], c["qs"], c["ks_"], c["vs_"], c["q_out"], c["k_out"], c["T"], c["iv"],
                                   c["n"], c["pre"], c["pos"], c["qw"], c["kw"], c["eps"], c["rope"], c["max_pos"],
                                   _cache(lib, c), c["shape"], c["ws"], c["bytes"], c["status"], 0, check=False)


SHARED = [  # what every call with a cache refuses
    (dict(T=-1), "INVALID_ARG"), (dict(n=-1), "INVALID_ARG"), (dict(iv=None), "INVALID_ARG"), (dict(iv=0x1004), "INVALID_ARG"),
    (dict(pre=None), "INVALID_ARG"), (dict(pre=0x1002), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"),
    (dict(ws=0x1080), "INVALID_ARG"), (dict(bytes=64), "INVALID_ARG"), (dict(status=0x1002), "INVALID_ARG"),
    (dict(pool_k=None), "INVALID_ARG"), (dict(pool_v=0x1008), "INVALID_ARG"), (dict(table=None), "INVALID_ARG"),
    (dict(max_blocks=0), "INVALID_ARG"), (dict(n_blocks=0), "INVALID_ARG"), (dict(pool="e4m3"), "INVALID_ARG"),
    (dict(pool="fp32"), "UNSUPPORTED"), (dict(n=4097), "UNSUPPORTED"), (dict(n_blocks=(1 << 20) + 1), "UNSUPPORTED"),
]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(q=None), "INVALID_ARG"), (dict(k=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"), (dict(q_out=None), "INVALID_ARG"),
    (dict(q=0x100008), "INVALID_ARG"), (dict(k_out=0x500004), "INVALID_ARG"), (dict(pos=0x1002), "INVALID_ARG"),
    (dict(rope=None), "INVALID_ARG"), (dict(rope=0x1008), "INVALID_ARG"), (dict(max_pos=0), "INVALID_ARG"),
    (dict(qw=0x1008), "INVALID_ARG"), (dict(kw=0x1004), "INVALID_ARG"), (dict(qw=0x1000, eps=0.0), "INVALID_ARG"),
    (dict(kw=0x1000, eps=NAN), "INVALID_ARG"), (dict(qw=0x1000, eps=INF), "INVALID_ARG"), (dict(qw=0x1000, eps=-1.0), "INVALID_ARG"),
    (dict(qs=1020), "INVALID_ARG"), (dict(qs=512), "INVALID_ARG"), (dict(ks_=260), "INVALID_ARG"), (dict(vs_=-256), "INVALID_ARG"),
    (dict(no_cache=True, k_out=None), "INVALID_ARG"), (dict(no_cache=True, pre=0x1001), "INVALID_ARG"),
    # overlaps: 8 tokens are 16,384 bytes of q, 4,096 of k and v
    (dict(q_out=0x103ff0), "INVALID_ARG"), (dict(q_out=0x200ff0), "INVALID_ARG"), (dict(q_out=0x300ff0), "INVALID_ARG"),
    (dict(k_out=0x200ff0), "INVALID_ARG"), (dict(k_out=0x103ff0), "INVALID_ARG"), (dict(k_out=0x300000), "INVALID_ARG"),
    (dict(k_out=0x403ff0), "INVALID_ARG"), (dict(q_out=0x100000, qs=1536), "INVALID_ARG"),
])
def test_norm_rope_refuses_on_the_host(lib, kw, code):
    assert norm_rope(lib, **kw) == getattr(lib.binding, "KEV_ERR_" + code)


def mass(lib, **kw):
    c = _defaults(lib, dict(q=0x1000, max_chunk=0, decay=1.0, mass=0x1000))
    c.update(kw)
    return lib.kev_attn_mass_paged(c["q"], c["T"], c["iv"], c["n"], c["pre"], c["max_chunk"], _cache(lib, c), c["decay"],
                                   c["mass"], c["shape"], c["ws"], c["bytes"], c["status"], 0, check=False)


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(q=None), "INVALID_ARG"), (dict(q=0x1008), "INVALID_ARG"), (dict(max_chunk=-1), "INVALID_ARG"),
    (dict(decay=-0.5), "INVALID_ARG"), (dict(decay=NAN), "INVALID_ARG"), (dict(decay=INF), "INVALID_ARG"),
    (dict(mass=None), "INVALID_ARG"), (dict(mass=0x1004), "INVALID_ARG"),
])
def test_mass_refuses_on_the_host(lib, kw, code):
    assert mass(lib, **kw) == getattr(lib.binding, "KEV_ERR_" + code)


def test_mass_workspace(lib):
    s = lib.make_shape(8, 2, 128, "bf16")
    sizes = [lib.kev_attn_mass_workspace_size(4, t, s) for t in (0, 1, 64, 1000, 2 ** 31 - 1)]
    assert sizes == sorted(sizes) and sizes[0] > 0 and sizes[-1] > 4 * 8 * (2 ** 31 - 1)
    assert mass(lib, bytes=lib.kev_attn_mass_workspace_size(2, 8, s) - 1) == lib.binding.KEV_ERR_INVALID_ARG
    assert lib.kev_attn_mass_workspace_size(4097, 4, s) == 0 and lib.kev_attn_mass_workspace_size(2, -1, s) == 0
    assert lib.kev_attn_mass_workspace_size(2, 4, lib.make_shape(8, 3, 128, "bf16")) == 0


EVICT = [
    (dict(n=-1), "INVALID_ARG"), (dict(keep=0), "INVALID_ARG"), (dict(max_blocks=0), "INVALID_ARG"), (dict(n_blocks=0), "INVALID_ARG"),
    (dict(table=None), "INVALID_ARG"), (dict(table=0x1002), "INVALID_ARG"), (dict(lens=None), "INVALID_ARG"),
    (dict(lens=0x1001), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"), (dict(ws=0x1080), "INVALID_ARG"), (dict(bytes=64), "INVALID_ARG"),
    (dict(status=0x1002), "INVALID_ARG"), (dict(kept=None), "INVALID_ARG"), (dict(kept=0x1002), "INVALID_ARG"),
    (dict(kept_lens=None), "INVALID_ARG"), (dict(kept_lens=0x2002), "INVALID_ARG"), (dict(n=4097), "UNSUPPORTED"),
    (dict(n_blocks=(1 << 20) + 1), "UNSUPPORTED"), (dict(max_blocks=(1 << 23) + 1), "UNSUPPORTED"),
    (dict(n=4096, keep=2 ** 31 - 1), "UNSUPPORTED"),
]


def select(lib, **kw):
    c = _defaults(lib, dict(mass=0x1000, lens=0x1000, active=None, keep=8, first=2, last=2, kept=0x1000, kept_lens=0x2000))
    c.update(kw)
    return lib.kev_select_paged(c["mass"], c["lens"], c["active"], c["n"], c["table"], c["max_blocks"], c["n_blocks"], c["keep"],
                                c["first"], c["last"], c["kept"], c["kept_lens"], c["shape"], c["ws"], c["bytes"], c["status"], 0,
                                check=False)


def compact(lib, **kw):
    c = _defaults(lib, dict(mass=0x1000, lens=0x1000, keep=8, kept=0x1000, kept_lens=0x2000))
    c.update(kw)
    return lib.kev_compact_paged(c["kept"], c["keep"], c["lens"], c["kept_lens"], c["n"],
                                 _cache(lib, c) if not c["no_cache"] else lib.binding.kev_paged_cache(), c["mass"], c["shape"],
                                 c["ws"], c["bytes"], c["status"], 0, check=False)


@pytest.mark.parametrize("kw,code", EVICT + [
    (dict(mass=None), "INVALID_ARG"), (dict(mass=0x1004), "INVALID_ARG"), (dict(first=-1), "INVALID_ARG"), (dict(last=-1), "INVALID_ARG"),
    (dict(first=5, last=4), "INVALID_ARG"), (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), "INVALID_ARG"), (dict(kept_lens=0x1000), "INVALID_ARG"),
])
def test_select_refuses_on_the_host(lib, kw, code):
    assert select(lib, **kw) == getattr(lib.binding, "KEV_ERR_" + code)


@pytest.mark.parametrize("kw,code", EVICT + [
    (dict(mass=0x1004), "INVALID_ARG"), (dict(pool_k=None), "INVALID_ARG"), (dict(pool_v=0x1008), "INVALID_ARG"),
    (dict(pool="e4m3"), "INVALID_ARG"), (dict(pool="fp32"), "UNSUPPORTED"), (dict(no_cache=True), "INVALID_ARG"),
])
def test_compact_refuses_on_the_host(lib, kw, code):
    assert compact(lib, **kw) == getattr(lib.binding, "KEV_ERR_" + code)


def test_evict_workspace(lib):
    s = lib.make_shape(8, 2, 128, "bf16")
    sizes = [lib.kev_evict_workspace_size(n, keep, s) for n, keep in ((0, 1), (1, 1), (32, 1024), (64, 100000))]
    assert sizes == sorted(sizes) and sizes[0] > 0 and sizes[2] >= 4 * 32 * 2 * 16
    assert lib.kev_evict_workspace_size(1, 0, s) == 0 and lib.kev_evict_workspace_size(-1, 8, s) == 0
    assert lib.kev_evict_workspace_size(4096, 2 ** 31 - 1, s) == 0


def logprobs(lib, **kw):
    c = dict(logits=0x1000, n=2, vocab=100, dtype="bf16", t=None, active=None, tokens=0x1000, lp=0x1000, ent=0x1000, top=3, tt=0x1000,
             tl=0x1000, status=None)
    c.update(kw)
    return lib.kev_logprobs(c["logits"], c["n"], c["vocab"], c["dtype"], c["t"], c["active"], c["tokens"], c["lp"], c["ent"], c["top"],
                            c["tt"], c["tl"], c["status"], 0, check=False)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), "INVALID_ARG"), (dict(logits=0x1008), "INVALID_ARG"), (dict(n=-1), "INVALID_ARG"), (dict(vocab=0), "INVALID_ARG"),
    (dict(t=0x1002), "INVALID_ARG"), (dict(tokens=None), "INVALID_ARG"), (dict(lp=None), "INVALID_ARG"), (dict(tokens=0x1001), "INVALID_ARG"),
    (dict(lp=0x1002), "INVALID_ARG"), (dict(ent=0x1002), "INVALID_ARG"), (dict(top=-1), "INVALID_ARG"), (dict(top=4, vocab=3), "INVALID_ARG"),
    (dict(tt=None), "INVALID_ARG"), (dict(tl=None), "INVALID_ARG"), (dict(tt=0x1002), "INVALID_ARG"), (dict(status=0x1001), "INVALID_ARG"),
    (dict(dtype=7), "UNSUPPORTED"), (dict(dtype=2), "UNSUPPORTED"), (dict(top=33), "UNSUPPORTED"), (dict(vocab=(1 << 30) + 1), "UNSUPPORTED"),
])
def test_logprobs_refuses_on_the_host(lib, kw, code):
    assert logprobs(lib, **kw) == getattr(lib.binding, "KEV_ERR_" + code)


def test_logprobs_of_no_rows(lib):
    assert logprobs(lib, n=0, logits=None, tokens=None, lp=None, ent=None, tt=None, tl=None) == 0


def test_launch_counts(lib):
    assert [lib.kev_launch_count(i) for i in (20, 21, 22, 23, 24, 25)] == [2, 4, 2, 2, 1, -1]
    assert lib.kev_status_string(12) != "unknown status"
