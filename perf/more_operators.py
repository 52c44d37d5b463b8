"""What a serving program does around the paged cache and the logits of a decode step, each operator beside its plain form.

* ``norm_rope``: the new tokens' query and key heads normalised (RMS, a learned weight per element) and rotated to their
  positions in one pass, out of the projection's rows, the keys and values going into the paged cache in its type;
* ``mass``: how much attention every cached position receives from the new tokens, added to what it received before;
* ``select``: the positions that a question keeps when its cache is cut to a budget: the first ones, the last ones and
  those with the most accumulated attention;
* ``compact``: the kept rows moved to the front of their question's pages;
* ``logprobs``: the log probability of a given token in every row of logits, the row's entropy and its likeliest tokens.

Lengths belong to a case and come from its own number ``draw``; the values come from the seed.
"""
import math

import numpy as np
import torch

own = False

PAGE = 128
E4M3_MAX = 448.0
THETA = 1e6
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _case(name, op, n=1, lens=(1, 1), prefix=(0, 0), heads=(32, 8), d=128, dtype="bf16", pool="bf16", fused=True, evicted=0,
          decay=1.0, keep=0, first=0, last=0, vocab=0, top=0, tempered=False, masked=False, draw=1):
    c = {"op": op, "n": n, "len_lo": lens[0], "len_hi": lens[1], "pre_lo": prefix[0], "pre_hi": prefix[1], "h_q": heads[0],
         "h_kv": heads[1], "d": d, "dtype": dtype, "pool": pool, "fused": fused, "evicted": evicted, "decay": decay,
         "keep": keep, "first": first, "last": last, "vocab": vocab, "top": top, "tempered": tempered, "masked": masked,
         "draw": draw}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step of 32 questions, Qwen3-8B heads: rows of a fused projection, caches that had rows evicted, so that
        # positions run ahead of the cached rows; the smallest call, all latency
        _case("norm rope decode", "norm_rope", 32, (1, 1), (64, 2400), pool="e4m3", evicted=500, draw=1),
        # the prompts of a batch before their attention
        _case("norm rope prompts", "norm_rope", 32, (64, 4096), draw=2),
        # attention received in one decode step over an 8-bit cache
        _case("mass decode e4m3", "mass", 32, (1, 1), (64, 2400), pool="e4m3", draw=3),
        # the same over long bf16 caches
        _case("mass decode long", "mass", 16, (1, 1), (2048, 32768), draw=4),
        # pieces of long prompts, every token of the piece a witness (Qwen2.5-7B heads)
        _case("mass chunk", "mass", 8, (128, 1024), (1, 8192), heads=(28, 4), draw=5),
        # what the last 32 tokens of long prompts look at: weights counted afresh, to cut each cache once after its prefill
        _case("mass window of witnesses", "mass", 8, (32, 32), (4000, 16384), pool="e4m3", decay=0.0, draw=6),
        # caches of a batch cut to 1024 rows
        _case("select batch", "select", 32, (200, 2400), keep=1024, first=4, last=128, draw=7),
        # long caches cut to 4096 rows
        _case("select long", "select", 16, (2048, 32768), keep=4096, first=4, last=512, draw=8),
        # and the moves of each
        _case("compact batch e4m3", "compact", 32, (200, 2400), pool="e4m3", keep=1024, first=4, last=128, draw=9),
        _case("compact long", "compact", 16, (2048, 32768), keep=4096, first=4, last=512, draw=10),
        # a decode step's logits over the Qwen3 vocabulary, each question with its own temperature: the sampled token's log
        # probability, the entropy and the 20 likeliest tokens
        _case("logprobs decode", "logprobs", 32, vocab=151936, top=20, tempered=True, draw=11),
        # the tokens of given texts scored
        _case("logprobs scoring", "logprobs", 4096, vocab=151936, top=5, draw=12),
    ]


_HEADS = [(28, 4), (32, 8), (16, 4), (8, 8), (16, 1), (12, 4), (8, 2)]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope", "mass", "mass", "select", "compact", "logprobs", "logprobs"])
    heads, d, tag = rng.choice(_HEADS), rng.choice([64, 128, 128]), rng.randrange(1 << 20)
    pool = rng.choice(["bf16", "e4m3"])
    n = _logint(rng, 1, 64)
    if op == "norm_rope":
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        return _case("", op, n, (1, _logint(rng, 1, 2048)), (0, _logint(rng, 1, 3000)), heads, d, dtype,
                     rng.choice(["e4m3", dtype]), rng.random() < 0.5, rng.choice([0, 700]), draw=tag)
    if op == "mass":
        decay = rng.choice([0.0, 1.0, 0.98])
        if rng.random() < 0.5:  # decode steps
            lo = _logint(rng, 1, 2048)
            return _case("", op, n, (1, rng.choice([1, 1, 2, 3])), (lo, lo * rng.choice([1, 2, 4])), heads, d, pool=pool,
                         decay=decay, draw=tag)
        top = _logint(rng, 5, 600)
        return _case("", op, _logint(rng, 1, 8), (max(1, top // 4), top), (0, _logint(rng, 1, 8192)), heads, d, pool=pool,
                     decay=decay, draw=tag)
    if op in ("select", "compact"):
        top = _logint(rng, 2, 16384)
        keep = _logint(rng, 1, top)
        first = min(rng.choice([0, 1, 4]), keep)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        return _case("", op, min(n, 32), (max(1, top // 8), top), heads=heads, d=d, dtype=dtype,
                     pool=rng.choice(["e4m3", dtype]), keep=keep, first=first, last=min(rng.choice([0, 16, 128]), keep - first),
                     draw=tag)
    vocab = rng.choice([151936, _logint(rng, 100, 160000)])
    return _case("", op, max(1, min(_logint(rng, 1, 4096), 4096 * 151936 // vocab // 2)), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                 vocab=vocab, top=rng.choice([0, 1, 5, 20, 32]), tempered=rng.random() < 0.5, masked=rng.random() < 0.3, draw=tag)


def _lengths(case):
    """(new tokens or cached positions, cached positions before them) of a case's questions, as numpy int64."""
    r = np.random.default_rng(case["draw"])

    def spread(lo, hi):
        a, b = math.log(lo + 1), math.log(hi + 1)
        return np.clip(np.rint(np.exp(r.uniform(a, b, case["n"])) - 1), lo, hi).astype(np.int64)

    lens = spread(case["len_lo"], case["len_hi"])
    return lens, spread(case["pre_lo"], case["pre_hi"])


def _cell(case):
    """Bytes of one cached row of one head: codes and scale, or the elements."""
    d = case["d"]
    return {"e4m3": d + 4, "bf16": 2 * d, "fp32": 4 * d}[case["pool"]]


def work(case):
    lens, pre = _lengths(case)
    t, hq, hkv, d = int(lens.sum()), case["h_q"], case["h_kv"], case["d"]
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "norm_rope":
        row = (hq + 2 * hkv) * d * e  # q, k and v of a token, and its row of the angle table
        return {"bytes": t * (row + hq * d * e + 2 * hkv * _cell(case)) + t * d * 4, "flops": 10 * t * (hq + hkv) * d}
    if case["op"] == "mass":
        pairs = int((lens * pre + lens * (lens + 1) // 2).sum())
        seen = int((lens + pre).sum())
        old = int(pre.sum()) if case["decay"] else 0
        return {"bytes": t * hq * d * e + seen * hkv * (_cell(case) + 4) + old * hkv * 4, "flops": 2 * d * hq * pairs}
    kept = int(np.minimum(lens, case["keep"]).sum())
    if case["op"] == "select":
        return {"bytes": 4 * hkv * (t + kept), "flops": hkv * t}
    if case["op"] == "compact":
        return {"bytes": hkv * kept * (2 * 2 * _cell(case) + 2 * 4 + 4), "flops": 0}
    n, v = case["n"], case["vocab"]
    return {"bytes": n * (v * e + 12 + 8 * case["top"]), "flops": 5 * n * v}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _quantise(x):
    """Rows of e4m3 codes and their scales: scale = max|x| / 448, code = x / scale rounded to nearest even."""
    scale = x.abs().amax(-1) / E4M3_MAX
    y = torch.where(scale[..., None] == 0, torch.zeros_like(x), x / scale[..., None])
    return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) + 7919 * case["draw"])
    host = np.random.default_rng([int(seed), case["draw"]])

    def rand(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    dt, n = _TYPES[case["dtype"]], case["n"]
    if case["op"] == "logprobs":
        v, top = case["vocab"], case["top"]
        x = rand(n, v, dtype=dt)
        x *= 2.5
        if case["masked"]:  # a grammar leaves some rows a few hundred tokens, a run of the first ones or one in fifty
            x[::3, min(v - 1, 200):] = -math.inf
            x[1::3] = x[1::3].masked_fill_(torch.rand(v, generator=g, device="cuda") > 0.02, -math.inf)
            x[1::3, v // 2] = 1.0
        s = {"logits": x, "tokens": torch.randint(0, min(v, 200) if case["masked"] else v, (n,), generator=g, device="cuda", dtype=torch.int32),
             "temperature": None, "logprobs": torch.empty(n, device="cuda"), "entropy": torch.empty(n, device="cuda"),
             "top_tokens": torch.empty(n, top, dtype=torch.int32, device="cuda"), "top_logprobs": torch.empty(n, top, device="cuda")}
        # half the tokens are likely ones, as sampled tokens are
        s["tokens"][::2] = x[::2].argmax(-1).int()
        if case["tempered"]:
            s["temperature"] = torch.rand(n, generator=g, device="cuda") * 1.2 + 0.2
            s["temperature"][::5] = 0.0  # greedy
        return {**s, "case": case}

    lens, pre = _lengths(case)
    hq, hkv, d = case["h_q"], case["h_kv"], case["d"]
    t = int(lens.sum())
    ends = np.cumsum(lens)
    s = {"case": case, "t": t, "max_chunk": int(lens.max()), "host_lens": lens, "host_pre": pre,
         "intervals": torch.from_numpy(np.stack([ends - lens, ends], 1).astype(np.int32)).cuda(),
         "prefix": torch.from_numpy(pre.astype(np.int32)).cuda(), "lens": torch.from_numpy(lens.astype(np.int32)).cuda()}
    pages = -(-(pre + lens) // PAGE)
    total, width = int(pages.sum()) + 3, int(pages.max())
    ids, at, table = host.permutation(total), 0, np.full((n, width), -1, np.int32)
    for i, p in enumerate(pages.tolist()):
        table[i, :p] = ids[at:at + p]
        at += p
    s.update(table=torch.from_numpy(table).cuda(), max_blocks=width, n_blocks=total, pool_k=None, pool_v=None, scale_k=None,
             scale_v=None)
    shape = (total, hkv, PAGE, d)
    if case["op"] != "select":
        if case["pool"] == "e4m3":
            s["pool_k"], s["scale_k"] = _quantise(rand(*shape))
            s["pool_v"], s["scale_v"] = _quantise(rand(*shape))
        else:
            s["pool_k"], s["pool_v"] = rand(*shape, dtype=_TYPES[case["pool"]]), rand(*shape, dtype=_TYPES[case["pool"]])
    if case["op"] != "norm_rope":
        # a few positions receive most of the attention
        s["mass"] = torch.exp(1.5 * rand(*shape[:3]))
    if case["op"] == "norm_rope":
        if case["fused"]:  # rows of one projection: the heads of q, of k and of v beside each other
            s["qkv"] = rand(t, (hq + 2 * hkv) * d, dtype=dt)
            s["qkv"] *= 3
            s["q"], s["k"], s["v"] = (s["qkv"][:, a * d:b * d] for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
        else:
            s["q"], s["k"], s["v"] = (rand(t, h * d, dtype=dt) for h in (hq, hkv, hkv))
        s["q_weight"], s["k_weight"] = ((1 + 0.3 * rand(d)).to(dt) for _ in range(2))
        s["q_out"] = torch.empty(t, hq, d, dtype=dt, device="cuda")
        start = pre + (host.integers(0, case["evicted"] + 1, n) if case["evicted"] else 0)
        s["start"] = torch.from_numpy(start.astype(np.int32)).cuda()
        s["max_pos"] = int((start + lens).max())
        w = THETA ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
        angle = torch.arange(s["max_pos"], device="cuda", dtype=torch.float64)[:, None] * w
        s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float()  # [max_pos, d / 2, 2], built once
    elif case["op"] == "mass":
        s["q"] = rand(t, hq, d, dtype=dt)
    else:
        keep = case["keep"]
        s["kept"] = torch.zeros(n, hkv, keep, dtype=torch.int32, device="cuda")
        s["kept_lens"] = torch.from_numpy(np.minimum(lens, keep).astype(np.int32)).cuda()
        if case["op"] == "compact":  # as a selection leaves them: the first ones, the last ones, and others between them
            score = torch.rand(n, hkv, width * PAGE, generator=g, device="cuda")
            pos = torch.arange(width * PAGE, device="cuda")
            size = s["lens"].long()[:, None, None]
            score[..., :case["first"]] = 2.0
            score = torch.where((pos >= size - case["last"]) & (pos < size), torch.full_like(score, 2.0), score)
            score = torch.where(pos < size, score, torch.full_like(score, -1.0))
            index = torch.argsort(score, dim=-1, descending=True, stable=True)[..., :keep]
            index = torch.where(torch.arange(index.shape[-1], device="cuda") < size, index, torch.full_like(index, width * PAGE))
            index = torch.sort(index, -1)[0]
            s["kept"][..., :index.shape[-1]] = torch.where(index < width * PAGE, index, torch.zeros_like(index)).int()
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def _own(s):
    import packed_question_isolated_gb300 as kev

    c = s["case"]
    n = c["n"]
    if "status" not in s:  # what a program keeps from step to step: status word, shape, cache handle, workspace
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if c["op"] != "logprobs":
            s["shape"] = kev.make_shape(c["h_q"], c["h_kv"], c["d"], c["dtype"])
            if c["op"] == "norm_rope":
                s["bytes"] = kev.kev_paged_workspace_size(n, s["t"], s["shape"])
            elif c["op"] == "mass":
                s["bytes"] = kev.kev_attn_mass_workspace_size(n, s["t"], s["shape"])
            else:
                s["bytes"] = kev.kev_evict_workspace_size(n, c["keep"], s["shape"])
            s["ws"] = torch.empty(s["bytes"], dtype=torch.uint8, device="cuda")
            if c["op"] != "select":
                s["cache"] = kev.make_paged_cache(s["pool_k"], s["pool_v"], s["table"], s["max_blocks"], s["n_blocks"], c["pool"],
                                                  s["scale_k"], s["scale_v"])
    if c["op"] == "logprobs":
        kev.kev_logprobs(s["logits"], n, c["vocab"], c["dtype"], s["temperature"], None, s["tokens"], s["logprobs"],
                         s["entropy"], c["top"], s["top_tokens"] if c["top"] else None,
                         s["top_logprobs"] if c["top"] else None, s["status"])
        return
    end = (s["shape"], s["ws"], s["bytes"], s["status"])
    if c["op"] == "norm_rope":
        kev.kev_norm_rope_paged(s["q"], s["k"], s["v"], s["q"].stride(0), s["k"].stride(0), s["v"].stride(0), s["q_out"], None,
                                s["t"], s["intervals"], n, s["prefix"], s["start"], s["q_weight"], s["k_weight"], EPS, s["rope"],
                                s["max_pos"], s["cache"], *end)
    elif c["op"] == "mass":
        kev.kev_attn_mass_paged(s["q"], s["t"], s["intervals"], n, s["prefix"], s["max_chunk"], s["cache"], c["decay"], s["mass"],
                                *end)
    elif c["op"] == "select":
        kev.kev_select_paged(s["mass"], s["lens"], None, n, s["table"], s["max_blocks"], s["n_blocks"], c["keep"], c["first"],
                             c["last"], s["kept"], s["kept_lens"], *end)
    else:
        kev.kev_compact_paged(s["kept"], c["keep"], s["lens"], s["kept_lens"], n, s["cache"], s["mass"], *end)


def _places(s, lens):
    """Question, packed place in it, and position of every new token."""
    i = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), lens.long(), output_size=s["t"])
    j = torch.arange(s["t"], device="cuda") - s["intervals"][i, 0]
    return i, j, s["prefix"][i].long() + j


def _stored(pool, scale, index):
    x = pool.view(torch.uint8)[index].view(torch.float8_e4m3fn).float() if scale is not None else pool[index].float()
    return x * scale[index][..., None] if scale is not None else x


def _plain_norm_rope(s):
    c = s["case"]
    hq, hkv, d, t = c["h_q"], c["h_kv"], c["d"], s["t"]
    i, j, pos = _places(s, s["lens"])
    turn = s["rope"][s["start"][i].long() + j][:, None]  # [t, 1, d / 2, 2]
    cos, sin = turn[..., 0], turn[..., 1]

    def one(x, h, w):
        x = x.float().view(t, h, d)
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        a, b = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    s["q_out"].copy_(one(s["q"], hq, s["q_weight"]))
    block, row = s["table"][i, pos // PAGE].long(), pos % PAGE
    for x, pool, scale in ((one(s["k"], hkv, s["k_weight"]), s["pool_k"], s["scale_k"]),
                           (s["v"].float().view(t, hkv, d), s["pool_v"], s["scale_v"])):
        if scale is None:
            pool[block, :, row] = x.to(pool.dtype)
        else:
            code, sc = _quantise(x)
            pool.view(torch.uint8)[block, :, row] = code.view(torch.uint8)
            scale[block, :, row] = sc


def _plain_mass(s):
    c = s["case"]
    n, hkv, d, g, tokens = c["n"], c["h_kv"], c["d"], c["h_q"] // c["h_kv"], s["max_chunk"]
    i, j, _ = _places(s, s["lens"])
    width = s["max_blocks"] * PAGE
    table = s["table"].long()
    k = _stored(s["pool_k"], s["scale_k"], table.clamp_min(0)).permute(0, 2, 1, 3, 4).reshape(n, hkv, width, d)
    q = torch.zeros(n, tokens, c["h_q"], d, device="cuda")
    q[i, j] = s["q"].float()
    q = q.view(n, tokens, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * tokens, d)
    score = (q @ k.transpose(-1, -2)).view(n, hkv, g, tokens, width) / math.sqrt(d)
    pre, size = s["prefix"].long(), (s["prefix"] + s["lens"]).long()
    step = torch.arange(tokens, device="cuda")
    key = torch.arange(width, device="cuda")
    seen = key <= pre[:, None, None] + step[:, None]
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    p = (score - score.amax(-1, keepdim=True)).exp_()
    p = p / p.sum(-1, keepdim=True)
    p = p * (step < s["lens"].long()[:, None])[:, None, None, :, None]  # questions with fewer tokens than the longest
    new = p.sum((2, 3))  # [n, h_kv, width]
    at = torch.arange(width, device="cuda") < size[:, None]
    q_of, u_of = at.nonzero(as_tuple=True)
    block, row = table[q_of, u_of // PAGE], u_of % PAGE
    old = s["mass"][block, :, row]  # [positions, h_kv]
    old = torch.where((u_of < pre[q_of])[:, None], old * c["decay"], torch.zeros_like(old)) if c["decay"] else 0.0
    s["mass"][block, :, row] = new[q_of, :, u_of] + old


def _plain_select(s):
    c = s["case"]
    n, hkv, keep = c["n"], c["h_kv"], c["keep"]
    width = s["max_blocks"] * PAGE
    x = s["mass"][s["table"].long().clamp_min(0)].permute(0, 2, 1, 3).reshape(n, hkv, width)
    pos = torch.arange(width, device="cuda")
    size = s["lens"].long()[:, None, None]
    bits = x.view(torch.int32).long()  # not negative: in the order of the values
    safe = (pos < c["first"]) | (pos >= size - c["last"])
    rank = torch.where(pos < size, torch.where(safe, torch.full_like(bits, 0x7fffffff), bits), torch.full_like(bits, -1))
    top = torch.topk((rank << 32) + (width - 1 - pos), min(keep, width), -1)[0]
    index = torch.where(top >= 0, width - 1 - (top & 0xffffffff), torch.full_like(top, width))
    index = torch.sort(index, -1)[0]
    live = index < width
    kept = s["kept"][..., :index.shape[-1]]
    kept.copy_(torch.where(live, index.int(), kept))
    s["kept_lens"].copy_(s["lens"].clamp_max(keep))


def _plain_compact(s):
    c = s["case"]
    q_of, j = (torch.arange(c["keep"], device="cuda") < s["kept_lens"][:, None]).nonzero(as_tuple=True)
    table, heads = s["table"].long(), torch.arange(c["h_kv"], device="cuda")
    u = s["kept"][q_of, :, j].long()  # [rows, h_kv]
    src = (table[q_of[:, None], u // PAGE], heads, u % PAGE)
    dst = (table[q_of, j // PAGE][:, None], heads, (j % PAGE)[:, None])
    for x in (s["pool_k"], s["pool_v"], s["scale_k"], s["scale_v"], s["mass"]):
        if x is not None:
            x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
            x[dst] = x[src]


def _plain_logprobs(s):
    c = s["case"]
    x, v, top = s["logits"].float(), c["vocab"], c["top"]
    best = x.amax(-1, keepdim=True)
    greedy = None
    z = x - best
    if s["temperature"] is not None:
        t = s["temperature"][:, None]
        greedy = t == 0
        z = z / torch.where(greedy, torch.ones_like(t), t)
    e = torch.exp(z)
    total = e.sum(-1, keepdim=True)
    part = torch.where(e > 0, e * z, torch.zeros_like(e)).sum(-1, keepdim=True)
    entropy, lse = total.log() - part / total, total.log()
    token = s["tokens"].long()[:, None]
    lp = z.gather(1, token) - lse
    if greedy is not None:  # all on the first of the largest
        argmax = torch.where(x == best, torch.arange(v, device="cuda"), v).amin(-1, keepdim=True)
        sure = torch.zeros_like(lp)
        lp = torch.where(greedy, torch.where(token == argmax, sure, sure - math.inf), lp)
        entropy = torch.where(greedy, sure, entropy)
    s["logprobs"].copy_(lp[:, 0])
    s["entropy"].copy_(entropy[:, 0])
    if not top:
        return
    bits = (s["logits"].float() + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7fffffff), bits)  # whole numbers in the order of the values
    key = (order << 32) + (v - 1 - torch.arange(v, device="cuda"))
    index = v - 1 - (torch.topk(key, top, -1)[0] & 0xffffffff)
    lp = z.gather(1, index) - lse
    if greedy is not None:
        lp = torch.where(greedy, torch.where(index == argmax, torch.zeros_like(lp), torch.full_like(lp, -math.inf)), lp)
    s["top_tokens"].copy_(index)
    s["top_logprobs"].copy_(lp)


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        _own(s)
    else:
        {"norm_rope": _plain_norm_rope, "mass": _plain_mass, "select": _plain_select, "compact": _plain_compact,
         "logprobs": _plain_logprobs}[op](s)
    if op == "logprobs":
        return {k: s[k] for k in ("logprobs", "entropy") + (("top_tokens", "top_logprobs") if c["top"] else ())}
    if op == "mass":
        return {"mass": s["mass"]}
    if op == "select":
        return {"kept": s["kept"], "kept_lens": s["kept_lens"]}
    r = {k: s[k] for k in ("pool_k", "pool_v", "scale_k", "scale_v") if s[k] is not None}
    r["q" if op == "norm_rope" else "mass"] = s["q_out" if op == "norm_rope" else "mass"]
    return r


# ---------------------------------------------------------------------------------------------------------------
# the definition in 64 bits, question by question and row by row
# ---------------------------------------------------------------------------------------------------------------
def _exact_logprobs(s):
    c = s["case"]
    out = {"logprobs": [], "entropy": [], "top_logprobs": []}
    for a in range(0, c["n"], 256):
        rows = slice(a, a + 256)
        x = s["logits"][rows].double()
        t = torch.ones(len(x), dtype=torch.float64, device="cuda") if s["temperature"] is None else s["temperature"][rows].double()
        greedy = t == 0
        y = torch.log_softmax(x / torch.where(greedy, torch.ones_like(t), t)[:, None], -1)
        first = torch.zeros_like(y).fill_(-math.inf)
        first.scatter_(1, (x == x.amax(-1, keepdim=True)).int().argmax(-1, keepdim=True), 0.0)
        y = torch.where(greedy[:, None], first, y)
        out["logprobs"].append(y.gather(1, s["tokens"][rows].long()[:, None])[:, 0])
        p = y.exp()
        out["entropy"].append(-torch.where(p > 0, p * y, torch.zeros_like(p)).sum(-1))
        if c["top"]:
            out["top_logprobs"].append(torch.sort(y, dim=-1, descending=True, stable=True)[0][:, :c["top"]])
    r = {"logprobs": torch.cat(out["logprobs"]), "entropy": torch.cat(out["entropy"])}
    if c["top"]:
        r.update(top_tokens=None, top_logprobs=torch.cat(out["top_logprobs"]))
    return r


def exact(case, seed):
    if case["op"] in ("select", "compact"):
        return None  # choices and copies: nothing is computed
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        return _exact_logprobs(s)
    lens, pre = s["host_lens"].tolist(), s["host_pre"].tolist()
    hq, hkv, d = case["h_q"], case["h_kv"], case["d"]
    host_table = s["table"].cpu().numpy()
    if case["op"] == "mass":
        mass = s["mass"].double()
        at = 0
        for i, (m, p) in enumerate(zip(lens, pre)):
            blocks = torch.from_numpy(host_table[i, :-(-(p + m) // PAGE)].astype(np.int64)).cuda()
            pool, scale = s["pool_k"], s["scale_k"]
            k = pool.view(torch.uint8)[blocks].view(torch.float8_e4m3fn).double() if scale is not None else pool[blocks].double()
            if scale is not None:
                k = k * scale[blocks].double()[..., None]
            k = k.permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :p + m]
            q = s["q"][at:at + m].double().view(m, hkv, hq // hkv, d)
            at += m
            got = torch.zeros(hkv, p + m, dtype=torch.float64, device="cuda")
            for a in range(0, m, 128):
                b = min(m, a + 128)
                z = torch.einsum("thgd,hud->htgu", q[a:b], k[:, :p + b]) / math.sqrt(d)
                late = torch.arange(p + b, device="cuda") > torch.arange(p + a, p + b, device="cuda")[:, None]
                z = z.masked_fill(late[None, :, None], -math.inf)
                got[:, :p + b] += torch.softmax(z, -1).sum((1, 2))
            flat = torch.arange(p + m, device="cuda")
            where = (blocks[flat // PAGE], slice(None), flat % PAGE)
            old = mass[where] * case["decay"]
            old[p:] = 0
            mass[where] = got.t() + old
        return {"mass": mass}
    # norm_rope
    w = THETA ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    start = s["start"].cpu().tolist()
    outs, at = [], 0
    scales = {k: s[k].double() if s[k] is not None else None for k in ("scale_k", "scale_v")}
    pools = {k: s[k].double() if s["scale_k"] is None else None for k in ("pool_k", "pool_v")}
    for i, (m, p) in enumerate(zip(lens, pre)):
        rows = slice(at, at + m)
        at += m
        angle = (torch.arange(start[i], start[i] + m, device="cuda", dtype=torch.float64)[:, None] * w)[:, None]

        def turned(x, h, weight):
            x = x[rows].double().view(m, h, d)
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.double()
            z = torch.polar(torch.ones_like(angle), angle) * torch.complex(x[..., :d // 2].contiguous(), x[..., d // 2:].contiguous())
            return torch.cat([z.real, z.imag], -1)

        outs.append(turned(s["q"], hq, s["q_weight"]))
        flat = torch.arange(p, p + m, device="cuda")
        blocks = s["table"][i].long()[flat // PAGE]
        for side, x in (("k", turned(s["k"], hkv, s["k_weight"])), ("v", s["v"][rows].double().view(m, hkv, d))):
            if s["scale_k"] is None:
                pools["pool_" + side][blocks, :, flat % PAGE] = x
            else:
                scales["scale_" + side][blocks, :, flat % PAGE] = x.abs().amax(-1) / E4M3_MAX
    r = dict(pools)
    r.update({k: x for k, x in scales.items() if x is not None})
    r["q"] = torch.cat(outs)
    return r
