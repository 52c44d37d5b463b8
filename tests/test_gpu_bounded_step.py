"""The operators together, as a serving program with a bounded cache calls them: the prompts' norms, rotation and cache
write, their attention and the attention each position received; the caches cut to a budget; then decode steps whose
positions run ahead of the cached rows, with the next token sampled and its log probability reported.  Every stage is
held to its float64 definition on what the stage before left on the device."""
import numpy as np
import pytest
import torch

import packed_question_isolated_gb300 as kev
from oracle import kev_oracle as O
from oracle import serve_oracle as S

from test_gpu_span import PAGE, TD, Span

pytestmark = pytest.mark.gpu
THETA, EPS, VOCAB = 1e6, 1e-6, 1000


class Serving:
    def __init__(self, pool, dtype, lens, keep, first, last, heads=(8, 2), d=64):
        self.pool, self.dtype, self.keep, self.first, self.last = pool, dtype, keep, first, last
        self.h_q, self.h_kv, self.d, self.n = *heads, d, len(lens)
        self.g = np.random.default_rng(5)
        s = Span(3, lens, [0] * len(lens), *heads, d, dtype, pool, width=-(-max(lens) // PAGE) + 1)
        pages = [-(-m // PAGE) + 1 for m in lens]  # room for the steps
        s.n_blocks = sum(pages)
        ids, at = self.g.permutation(s.n_blocks), 0
        s.table[:] = -1
        for i, m in enumerate(pages):
            s.table[i, :m] = ids[at:at + m]
            at += m
        shape = (s.n_blocks, self.h_kv, PAGE, d)
        s.pools = [(torch.zeros(shape, device="cuda").to(TD[pool]), torch.zeros(shape[:3], device="cuda") if pool == "e4m3" else None)
                   for _ in range(2)]
        s.to_device()
        self.s = s
        self.mass = torch.full(shape[:3], float("nan"), device="cuda")
        self.w = [torch.from_numpy(1 + 0.2 * self.g.standard_normal(d, dtype=np.float32)).to(TD[dtype]).cuda() for _ in range(2)]
        self.max_pos = max(lens) + 40
        self.rope = torch.empty(self.max_pos, d // 2, 2, device="cuda")
        kev.kev_rope_table(self.rope, self.max_pos, d, THETA)
        self.seen = torch.zeros(self.n, dtype=torch.int32, device="cuda")   # tokens so far
        self.lens = torch.zeros(self.n, dtype=torch.int32, device="cuda")   # cached rows
        self.kept = torch.zeros(self.n, self.h_kv, keep, dtype=torch.int32, device="cuda")
        self.kept_lens = torch.zeros(self.n, dtype=torch.int32, device="cuda")
        self.head = torch.from_numpy(self.g.standard_normal((self.h_q * d, VOCAB), dtype=np.float32) / 8).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def round(self, new):
        """new[i] tokens of question i through the layer; returns the logits of every question's last token."""
        n, T, sh = self.n, sum(new), self.s.shape
        ends = np.cumsum(new)
        iv = torch.from_numpy(np.stack([ends - new, ends], 1).astype(np.int32)).cuda()
        self.qkv = torch.from_numpy(self.g.standard_normal((T, (self.h_q + 2 * self.h_kv) * self.d), dtype=np.float32)).to(TD[self.dtype]).cuda()
        q, k, v = (self.qkv[:, a * self.d:] for a in (0, self.h_q, self.h_q + self.h_kv))
        self.q, self.out = (torch.empty(T, self.h_q, self.d, dtype=TD[self.dtype], device="cuda") for _ in range(2))
        size = max(kev.kev_paged_workspace_size(n, T, sh), kev.kev_attn_mass_workspace_size(n, T, sh))
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        stride = self.qkv.stride(0)
        kev.kev_norm_rope_paged(q, k, v, stride, stride, stride, self.q, None, T, iv, n, self.lens, self.seen, *self.w, EPS, self.rope,
                                self.max_pos, self.s.cache, sh, ws, size, self.status)
        kev.kev_chunk_attn_paged(self.q, None, None, T, iv, n, self.lens, max(new), self.s.cache, 0, 0, self.out, sh, ws, size, self.status)
        kev.kev_attn_mass_paged(self.q, T, iv, n, self.lens, max(new), self.s.cache, 1.0, self.mass, sh, ws, size, self.status)
        last = torch.from_numpy(ends - 1).cuda()
        return iv, self.out[last].float().view(n, -1) @ self.head

    def cut(self):
        nb = kev.kev_evict_workspace_size(self.n, self.keep, self.s.shape)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        c = self.s.cache
        kev.kev_select_paged(self.mass, self.lens, None, self.n, self.s.tab, c.max_blocks, c.n_blocks, self.keep, self.first, self.last,
                             self.kept, self.kept_lens, self.s.shape, ws, nb, self.status)
        kev.kev_compact_paged(self.kept, self.keep, self.lens, self.kept_lens, self.n, c, self.mass, self.s.shape, ws, nb, self.status)
        self.lens.copy_(self.kept_lens)

    def caches(self, lens):
        self.s.prefix, self.s.lens = list(lens), [0] * self.n
        return self.s.caches()

    def masses(self, lens):
        x = self.mass.cpu().numpy()
        return [x[np.maximum(self.s.table[i, :-(-m // PAGE)], 0)].transpose(0, 2, 1).reshape(-1, self.h_kv)[:m] for i, m in enumerate(lens)]


@pytest.mark.parametrize("pool,dtype", [("bf16", "bf16"), ("e4m3", "bf16"), ("fp32", "fp32")])
def test_a_bounded_cache_through_prompts_and_steps(pool, dtype):
    lens = [300, 150, 90, 260]
    s = Serving(pool, dtype, lens, keep=140, first=4, last=20)
    before, new = [0] * 4, lens
    for step in range(6):
        old_cache, old_mass = s.caches(before), s.masses(before)
        iv, logits = s.round(new)
        assert kev.kev_read_status(s.status) == 0
        now = [b + m for b, m in zip(before, new)]
        cache, mass = s.caches(now), s.masses(now)
        iv = iv.cpu().numpy()
        for i in range(4):  # the rows before stay, the new keys are normalised and turned to the tokens' own positions
            for x, y in zip(cache[i], old_cache[i]):
                np.testing.assert_array_equal(x[:before[i]], y)
            rows = slice(iv[i, 0], iv[i, 1])
            k = s.qkv[rows, s.h_q * s.d:(s.h_q + s.h_kv) * s.d].float().cpu().numpy().reshape(-1, s.h_kv, s.d)
            want = S.norm_rope(k, s.w[1].float().cpu().numpy(), EPS, int(s.seen[i]) + np.arange(new[i]), THETA)
            step_size = {"fp32": 2.0 ** -16, "bf16": 2.0 ** -8 + 2.0 ** -16, "e4m3": 2.0 ** -4}[pool]
            assert (np.abs(cache[i][0][before[i]:] - want) <= step_size * np.abs(want) + 2.0 ** -10 * np.abs(want).max()).all()
        q = s.q.float().cpu().numpy().astype(np.float64)
        ref, size = O.span_attention(q, [k for k, _ in cache], [v for _, v in cache], before, iv, 0, 0)
        got = s.out.float().cpu().numpy()
        assert (np.abs(got - ref) <= (2.0 ** -7 + 2.0 ** -11 if dtype == "bf16" else 2.0 ** -14) * size).all()
        want, _ = S.attn_mass(q, [k for k, _ in cache], before, iv, [np.concatenate([o, np.zeros((m, s.h_kv))]) for o, m in zip(old_mass, new)], 1.0)
        for x, y in zip(mass, want):
            assert (np.abs(x - y) <= 2.0 ** -10 * y).all()
        s.lens += torch.tensor(new, dtype=torch.int32, device="cuda")
        s.seen += torch.tensor(new, dtype=torch.int32, device="cuda")
        if step % 2 == 0:
            s.cut()
            assert kev.kev_read_status(s.status) == 0
            kept, kept_lens = s.kept.cpu().numpy(), s.kept_lens.cpu().numpy()
            assert kept_lens.tolist() == [min(m, 140) for m in now]
            small, small_mass = s.caches(kept_lens.tolist()), s.masses(kept_lens.tolist())
            for i, m in enumerate(kept_lens):
                np.testing.assert_array_equal(kept[i, :, :m], S.select(mass[i], 140, 4, 20))
                for h in range(s.h_kv):
                    np.testing.assert_array_equal(small_mass[i][:, h], mass[i][kept[i, h, :m], h])
                    for x, y in zip(small[i], cache[i]):
                        np.testing.assert_array_equal(x[:, h], y[kept[i, h, :m], h])
            now = kept_lens.tolist()
        # the next tokens, and how likely they were
        temperature = torch.tensor([0.0, 0.7, 1.0, 1.5], device="cuda")
        uniforms = torch.from_numpy(s.g.random(4, dtype=np.float32)).cuda()
        live = torch.ones(4, dtype=torch.uint8, device="cuda")
        tokens = torch.zeros(4, dtype=torch.int32, device="cuda")
        kev.kev_sample(logits, 4, VOCAB, "fp32", temperature, uniforms, live, tokens, s.status)
        lp, ent, tl = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda"), torch.zeros(4, 3, device="cuda")
        tt = torch.zeros(4, 3, dtype=torch.int32, device="cuda")
        kev.kev_logprobs(logits, 4, VOCAB, "fp32", temperature, live, tokens, lp, ent, 3, tt, tl, s.status)
        assert kev.kev_read_status(s.status) == 0
        wlp, went, wtt, wtl = S.logprobs(logits.cpu().numpy(), temperature.cpu().numpy(), tokens.cpu().numpy(), 3)
        assert np.isfinite(wlp).all() and wlp[0] == 0  # a sampled token is possible, the greedy one certain
        np.testing.assert_allclose(lp.cpu().numpy(), wlp, atol=1e-4)
        np.testing.assert_allclose(ent.cpu().numpy(), went, atol=1e-3)
        np.testing.assert_array_equal(tt.cpu().numpy(), wtt)
        before, new = now, [1, 1, 1, 1] if step != 2 else [1, 3, 1, 2]
