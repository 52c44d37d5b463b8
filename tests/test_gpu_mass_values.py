"""kev_attn_mass_paged on infinite keys and rows of NaN, against the float64 definition.

Tolerances as derived in test_gpu_mass.py, S taken over the finite keys."""
import numpy as np
import pytest
import torch

from test_gpu_mass import Mass
from test_gpu_span import PAGE

pytestmark = pytest.mark.gpu


def definition(m, decay, scale=None):
    """New mass of every question, keys of an infinity among them, and the largest finite sum of |q_e k_e| * scale."""
    q = m.q.float().cpu().numpy().astype(np.float64)
    scale = 1 / np.sqrt(m.d) if scale is None else scale
    out, top = [], 0.0
    for i, (k, _) in enumerate(m.caches()):
        p, (b, e) = m.prefix[i], m.intervals[i]
        new = np.zeros((p + e - b, m.h_kv))
        for t in range(b, e):
            n = p + t - b + 1
            for h in range(m.h_q):
                g = h // (m.h_q // m.h_kv)
                with np.errstate(invalid="ignore"):
                    z = (k[:n, g] * q[t, h]).sum(-1) * scale
                fine = np.isfinite(z)
                if fine.any():
                    top = max(top, float((np.abs(k[:n, g][fine]) @ np.abs(q[t, h])).max()) * scale)
                w = np.exp(z - z.max())
                new[:n, g] += w / w.sum()
        if decay:
            new[:p] += decay * m.positions(m.old, i)[:p]
        out.append(new)
    return out, top


def near_definition(m, decay=1.0):
    want, top = definition(m, decay)
    rel = ((8 * (m.d + 8) + 8) * top + 16 + max(m.lens) * m.h_q / m.h_kv) * 2.0 ** -24
    got = m.mass.cpu().numpy()
    for i, y in enumerate(want):
        x = m.positions(got, i).astype(np.float64)
        assert np.isfinite(y).all()
        assert (np.abs(x - y) <= rel * np.abs(y) + 1e-30).all(), (i, np.argwhere(~(np.abs(x - y) <= rel * np.abs(y) + 1e-30))[:5].tolist())
    return want


# tokens that all see a key of the first page (whole row tiles, and one that the question ends in), few rows, one page alone
BATCHES = [([40, 3], [300, 130], 0), ([18, 36], [128, 250], 0), ([1, 1], [300, 5], 1), ([90], [0], 0), ([150], [128], 0)]


@pytest.mark.parametrize("batch", range(len(BATCHES)))
@pytest.mark.parametrize("dtype,pool", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32"), ("fp32", "e4m3")])
@pytest.mark.parametrize("h_q,h_kv", [(14, 2), (6, 2), (15, 3), (8, 2), (10, 1)])
def test_an_infinite_key_of_minus_infinite_scores_receives_nothing(h_q, h_kv, dtype, pool, batch):
    """q of one sign in the element that is infinite: the score is -infinity, the weight 0, every other mass finite."""
    lens, prefix, max_chunk = BATCHES[batch]
    m = Mass(30 + batch, lens, prefix, h_q, h_kv, 64, dtype, pool)
    m.q.copy_(m.q.abs() + 0.125)
    k, ks = m.pools[0]
    for i in range(len(lens)):
        n = prefix[i] + lens[i]
        for u in {3, n // 2, n - 2} & set(range(1, n)):
            b = int(m.table[i, u // PAGE])
            if pool == "e4m3":  # codes of -1 under an infinite scale
                k.view(torch.uint8)[b, 0, u % PAGE] = 0xb8
                ks[b, 0, u % PAGE] = float("inf")
            else:
                k[b, 0, u % PAGE, 5] = float("-inf")
    m.call(0.5, max_chunk)
    m.ok()
    near_definition(m, 0.5)


@pytest.mark.parametrize("bad", ["q nan", "q inf", "k inf", "k nan"])
@pytest.mark.parametrize("dtype,pool", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32"), ("fp32", "e4m3")])
@pytest.mark.parametrize("h_q,h_kv,tokens,prefix,max_chunk", [(2, 2, 11, 164, 0), (6, 2, 5, 60, 5), (4, 1, 4, 127, 4), (8, 1, 2, 15000, 2),
                                                              (6, 2, 60, 300, 0), (1, 1, 16, 0, 16)])
def test_a_row_without_weights_does_not_reach_positions_that_it_does_not_see(h_q, h_kv, tokens, prefix, max_chunk, dtype, pool, bad):
    """One row is NaN throughout, of a NaN or of an infinite score; the positions after it are as the later rows make them."""
    m = Mass(50, [tokens], [prefix], h_q, h_kv, 64, dtype, pool)
    t = tokens // 2 if max_chunk != 2 else 0
    if bad[0] == "q":
        m.q[t, 1 % h_q] = float(bad[2:])
        want = np.zeros((prefix + tokens, h_kv), bool)
        want[:prefix + t + 1, (1 % h_q) // (h_q // h_kv)] = True
    else:  # a key of a new token: the rows from that token on see it, those before do not
        k, ks = m.pools[0]
        b, row = int(m.table[0, (prefix + t) // PAGE]), (prefix + t) % PAGE
        m.q.copy_(m.q.abs() + 0.125)
        if pool == "e4m3":
            k.view(torch.uint8)[b, 0, row] = 0x7f if bad == "k nan" else 0x38  # NaN, 1
            ks[b, 0, row] = float(bad[2:])
        else:
            k[b, 0, row, 3] = float(bad[2:])
        want = np.zeros((prefix + tokens, h_kv), bool)
        want[:, 0] = True
    m.call(0.5, max_chunk)
    m.ok()
    got = m.positions(m.mass.cpu().numpy(), 0)
    assert (np.isnan(got) == want).all(), np.argwhere(np.isnan(got) != want)[:5].tolist()
    if bad[0] == "q":
        with np.errstate(invalid="ignore"):
            ref, top = definition(m, 0.5)
        rel = ((8 * 72 + 8) * top + 16 + tokens * h_q / h_kv) * 2.0 ** -24
        assert (np.abs(got - ref[0]) <= rel * ref[0] + 1e-30)[~want].all()
