"""The serving operators around the paged cache, as a user's program calls them, each beside its plain form.

* ``write`` / ``read``: the K/V rows of a chunk of every question into an 8-bit (e4m3) paged cache with one fp32 scale
  per row and head, and back out of it;
* ``chunk``: the new tokens of every question (one each in a decode step, many in a chunked prefill, both in a mixed
  batch) written to the paged cache and attending over it, with or without a sliding window and sink positions;
* ``window``: packed prefill attention under a sliding window with sink positions that stay visible.

Lengths belong to a case and come from its own number ``draw``; the values come from the seed.
"""
import math

import numpy as np
import torch

own = False

PAGE = 128
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _case(name, op, n, lens, prefix=(0, 0), heads=(32, 8), d=128, dtype="bf16", pool="e4m3", window=0, sinks=0, singles=0,
          draw=1):
    c = {"op": op, "n": n, "len_lo": lens[0], "len_hi": lens[1], "pre_lo": prefix[0], "pre_hi": prefix[1], "h_q": heads[0],
         "h_kv": heads[1], "d": d, "dtype": dtype, "pool": pool, "window": window, "sinks": sinks, "singles": singles,
         "draw": draw}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step's new K/V rows of 32 live questions: the smallest call, all latency
        _case("write one row each", "write", 32, (1, 1), (64, 2400), draw=1),
        # the prompts of a Qwen3-8B-shaped layer going into the 8-bit cache after their prefill
        _case("write prompts", "write", 32, (64, 4096), draw=2),
        # cached questions read back whole (to move them, or for a kernel that wants bf16 rows)
        _case("read prompts", "read", 64, (64, 8192), draw=3),
        # Qwen3-8B-shaped decode step, 32 live questions of 64 to 2400 cached positions, 8-bit cache
        _case("decode e4m3", "chunk", 32, (1, 1), (64, 2400), draw=4),
        # decode over long caches in bf16: 16 questions of up to 32 Ki positions
        _case("decode long bf16", "chunk", 16, (1, 1), (2048, 32768), pool="bf16", draw=5),
        # decode of a windowed layer: only the window and the sinks of each cache are read (28/4 heads)
        _case("decode window e4m3", "chunk", 64, (1, 1), (1024, 16384), heads=(28, 4), window=1024, sinks=4, draw=6),
        # later pieces of long prompts over a bf16 cache, Qwen2.5-7B heads
        _case("chunk bf16", "chunk", 8, (128, 1024), (1, 8192), heads=(28, 4), pool="bf16", draw=7),
        # the same over an 8-bit cache, Qwen3-8B heads, ragged sizes
        _case("chunk e4m3", "chunk", 8, (100, 600), (500, 16000), draw=8),
        # a scheduler's round: four prompts' pieces beside sixty decoding questions
        _case("mixed bf16", "chunk", 4, (256, 512), (64, 4096), pool="bf16", singles=60, draw=9),
        # eight prompts of at most 2048 tokens in one pass (Qwen2.5-7B heads), windowed layer
        _case("window prompts", "window", 8, (256, 2048), heads=(28, 4), window=512, sinks=4, draw=10),
        # long documents: the largest pass
        _case("window long", "window", 4, (4096, 16384), window=2048, sinks=16, draw=11),
        # many short questions through small heads
        _case("window d64", "window", 64, (16, 700), heads=(16, 4), d=64, window=128, sinks=1, draw=12),
    ]


_HEADS = [(28, 4), (32, 8), (16, 4), (8, 8), (16, 1), (12, 4), (8, 2)]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["write", "read", "decode", "decode", "chunk", "chunk", "window", "window"])
    heads, d = rng.choice(_HEADS), rng.choice([64, 128, 128])
    pool = rng.choice(["bf16", "e4m3"])
    wide = rng.random() < 0.5
    window, sinks = (_logint(rng, 16, 4096), rng.choice([0, 1, 4, 130])) if wide else (0, 0)
    tag = rng.randrange(1 << 20)
    n = _logint(rng, 1, 64)
    if kind in ("write", "read"):
        return _case("", kind, n, (1, _logint(rng, 1, 4096)), (0, _logint(rng, 1, 3000)), heads, d,
                     rng.choice(["bf16", "bf16", "fp32"]), "e4m3", draw=tag)
    if kind == "decode":
        lo = _logint(rng, 1, 2048)
        return _case("", "chunk", n, (1, rng.choice([1, 1, 2, 3])), (lo, lo * rng.choice([1, 2, 4])), heads, d, "bf16", pool,
                     window, sinks, draw=tag)
    if kind == "chunk":
        n = _logint(rng, 1, 8)
        top = _logint(rng, 5, 700)
        return _case("", "chunk", n, (max(1, top // 4), top), (0, _logint(rng, 1, 8192)), heads, d, "bf16", pool, window, sinks,
                     rng.choice([0, 0, 9]), tag)
    top = _logint(rng, 2, 4096)
    return _case("", "window", _logint(rng, 1, 8), (max(1, top // 8), top), heads=heads, d=d, pool="bf16",
                 window=window or _logint(rng, 16, 2048), sinks=sinks, draw=tag)


def _lengths(case):
    """(lengths, prefix lengths) of a case's questions, as numpy int64."""
    r = np.random.default_rng(case["draw"])

    def spread(lo, hi, n):
        a, b = math.log(lo + 1), math.log(hi + 1)
        return np.clip(np.rint(np.exp(r.uniform(a, b, n)) - 1), lo, hi).astype(np.int64)

    lens = spread(case["len_lo"], case["len_hi"], case["n"])
    lens = r.permutation(np.concatenate([lens, np.ones(case["singles"], np.int64)]))
    pre = spread(case["pre_lo"], case["pre_hi"], len(lens)) if case["op"] != "window" else np.zeros(len(lens), np.int64)
    return lens, pre


def _visible(case, lens, pre):
    """(query, key) pairs that see each other, and the cached positions of the prefixes that some new token sees."""
    w, s = case["window"] or 1 << 40, case["sinks"]
    pairs, old = 0, 0
    for n, p in zip(lens.tolist(), pre.tolist()):
        pos = np.arange(p, p + n)
        first = np.maximum(0, pos - w + 1)
        pairs += int((pos - first + 1 + np.minimum(first, s)).sum())
        f = max(0, p - w + 1)
        old += (p - min(f, p)) + min(f, s, p)
    return pairs, old


def work(case):
    lens, pre = _lengths(case)
    t, hq, hkv, d = int(lens.sum()), case["h_q"], case["h_kv"], case["d"]
    e = 4 if case["dtype"] == "fp32" else 2
    cell = d + 4 if case["pool"] == "e4m3" else 2 * d  # one cached row of one head: codes and scale, or bf16
    rows = 2 * t * hkv * d * e  # the new K and V rows
    if case["op"] in ("write", "read"):
        return {"bytes": rows + 2 * t * hkv * cell, "flops": 2 * t * hkv * d}
    pairs, old = _visible(case, lens, pre)
    b = rows + 2 * t * hq * d * e
    if case["op"] == "chunk":
        b += 2 * (t + old) * hkv * cell
    return {"bytes": b, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _quantise(x):
    """Rows of e4m3 codes and their scales: scale = max|x| / 448, code = x / scale rounded to nearest even."""
    x = x.float()
    scale = x.abs().amax(-1) / E4M3_MAX
    y = torch.where(scale[..., None] == 0, torch.zeros_like(x), x / scale[..., None])
    return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    lens, pre = _lengths(case)
    n, t = len(lens), int(lens.sum())
    hq, hkv, d = case["h_q"], case["h_kv"], case["d"]
    dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(int(seed) + 7919 * case["draw"])
    host = np.random.default_rng([int(seed), case["draw"]])

    def rand(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    ends = np.cumsum(lens)
    intervals = np.stack([ends - lens, ends], 1).astype(np.int32)
    s = {"case": case, "n": n, "t": t, "max_chunk": int(lens.max()), "host_lens": lens, "host_pre": pre,
         "intervals": torch.from_numpy(intervals).cuda(), "prefix": torch.from_numpy(pre.astype(np.int32)).cuda(),
         "k": rand(t, hkv, d), "v": rand(t, hkv, d)}
    if case["op"] in ("chunk", "window"):
        s["q"] = rand(t, hq, d)
        s["out"] = torch.empty_like(s["q"])
    else:
        s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    if case["op"] != "window":
        pages = -(-(pre + lens) // PAGE)
        total, width = int(pages.sum()) + 3, int(pages.max())
        ids, at, table = host.permutation(total), 0, np.full((n, width), -1, np.int32)
        for i, p in enumerate(pages.tolist()):
            table[i, :p] = ids[at:at + p]
            at += p
        s.update(table=torch.from_numpy(table).cuda(), max_blocks=width, n_blocks=total)
        shape = (total, hkv, PAGE, d)
        if case["pool"] == "e4m3":
            s["pool_k"], s["scale_k"] = _quantise(rand(*shape))
            s["pool_v"], s["scale_v"] = _quantise(rand(*shape))
        else:
            s["pool_k"], s["pool_v"] = rand(*shape, dtype=torch.bfloat16), rand(*shape, dtype=torch.bfloat16)
            s["scale_k"] = s["scale_v"] = None
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def _own(s):
    import packed_question_isolated_gb300 as kev

    c = s["case"]
    if "ws" not in s:  # what a program keeps from step to step: shape, cache handle, workspace, status word
        s["shape"] = kev.make_shape(c["h_q"], c["h_kv"], c["d"], c["dtype"])
        s["bytes"] = kev.kev_paged_workspace_size(s["n"], s["t"], s["shape"])
        s["ws"] = torch.empty(s["bytes"], dtype=torch.uint8, device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if c["op"] != "window":
            s["cache"] = kev.make_paged_cache(s["pool_k"], s["pool_v"], s["table"], s["max_blocks"], s["n_blocks"], c["pool"],
                                              s["scale_k"], s["scale_v"])
    end = (s["shape"], s["ws"], s["bytes"], s["status"])
    if c["op"] == "write":
        kev.kev_paged_write(s["k"], s["v"], s["t"], s["intervals"], s["n"], s["prefix"], s["cache"], *end)
    elif c["op"] == "read":
        kev.kev_paged_read(s["k_out"], s["v_out"], s["t"], s["intervals"], s["n"], s["prefix"], s["cache"], *end)
    elif c["op"] == "chunk":
        kev.kev_chunk_attn_paged(s["q"], s["k"], s["v"], s["t"], s["intervals"], s["n"], s["prefix"], s["max_chunk"],
                                 s["cache"], c["window"], c["sinks"], s["out"], *end)
    else:
        kev.kev_prefill_attn_window(s["q"], s["k"], s["v"], s["t"], s["intervals"], s["n"], c["window"], c["sinks"], s["out"],
                                    *end)


def _places(s):
    """Question, position, cache block and row of every packed token."""
    lens = (s["intervals"][:, 1] - s["intervals"][:, 0]).long()
    i = torch.repeat_interleave(torch.arange(s["n"], device="cuda"), lens, output_size=s["t"])
    j = torch.arange(s["t"], device="cuda") - s["intervals"][i, 0]
    pos = s["prefix"][i].long() + j
    return i, j, pos, s["table"][i, pos // PAGE].long() if "table" in s else None, pos % PAGE


def _plain_write(s):
    _, _, _, block, row = _places(s)
    for x, pool, scale in ((s["k"], s["pool_k"], s["scale_k"]), (s["v"], s["pool_v"], s["scale_v"])):
        if scale is None:
            pool[block, :, row] = x.to(pool.dtype)
        else:
            code, sc = _quantise(x)
            pool.view(torch.uint8)[block, :, row] = code.view(torch.uint8)
            scale[block, :, row] = sc


def _stored(pool, scale, index):
    x = pool.view(torch.uint8)[index].view(torch.float8_e4m3fn).float() if scale is not None else pool[index].float()
    return x * scale[index][..., None] if scale is not None else x


def _plain_chunk(s):
    c = s["case"]
    _plain_write(s)
    i, j, pos, _, _ = _places(s)
    n, hkv, d, g = s["n"], c["h_kv"], c["d"], c["h_q"] // c["h_kv"]
    tokens, width = s["max_chunk"], s["table"].shape[1] * PAGE
    table = s["table"].long().clamp_min(0)
    # [n, h_kv, width, d]: every question's cache, padded to the longest
    k, v = (_stored(p, sc, table).permute(0, 2, 1, 3, 4).reshape(n, hkv, width, d)
            for p, sc in ((s["pool_k"], s["scale_k"]), (s["pool_v"], s["scale_v"])))
    q = torch.zeros(n, tokens, c["h_q"], d, device="cuda")
    q[i, j] = s["q"].float()
    q = q.view(n, tokens, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * tokens, d)
    score = (q @ k.transpose(-1, -2)).view(n, hkv, g, tokens, width) / math.sqrt(d)
    at = s["prefix"].long()[:, None, None] + torch.arange(tokens, device="cuda")[None, :, None]
    key = torch.arange(width, device="cuda")
    seen = key <= at
    if c["window"]:
        seen &= (key > at - c["window"]) | (key < c["sinks"])
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    p = (score - score.amax(-1, keepdim=True)).exp_()
    o = (p.view(n, hkv, g * tokens, width) @ v).view(n, hkv, g, tokens, d) / p.sum(-1, keepdim=True)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(n, tokens, c["h_q"], d)[i, j])


def _plain_window(s):
    c = s["case"]
    i, j, pos, _, _ = _places(s)
    t, hkv, d, g, w, sinks = s["t"], c["h_kv"], c["d"], c["h_q"] // c["h_kv"], c["window"], c["sinks"]
    size = 256  # queries a block; each block looks at the packed positions its window can reach
    blocks = -(-t // size)
    pad = blocks * size
    first = s["intervals"][i, 0].long()
    q = torch.zeros(pad, c["h_q"], d, device="cuda")
    q[:t] = s["q"].float()
    q = q.view(blocks, size, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(blocks, hkv, g * size, d)
    at = torch.arange(pad, device="cuda").view(blocks, size)
    begin = torch.zeros(pad, dtype=torch.long, device="cuda")
    begin[:t] = first
    begin = begin.view(blocks, size)
    reach = torch.arange(1 - w, size, device="cuda")
    key = at[:, :1] + reach  # [blocks, w - 1 + size]
    inside = key.clamp(0, t - 1)
    k, v = s["k"].float()[inside].permute(0, 2, 1, 3), s["v"].float()[inside].permute(0, 2, 1, 3)
    near = (q @ k.transpose(-1, -2)).view(blocks, hkv, g, size, -1) / math.sqrt(d)
    key, here, start = key[:, None, :], at[:, :, None], begin[:, :, None]
    near.masked_fill_(~((key <= here) & (key > here - w) & (key >= start))[:, None, None], -math.inf)
    # the sinks of every token's own question, where they lie before its window
    far = begin[:, :, None] + torch.arange(sinks, device="cuda")
    ok = (far <= here - w) & (far < t)
    ks, vs = s["k"].float()[far.clamp_max(t - 1)], s["v"].float()[far.clamp_max(t - 1)]  # [blocks, size, sinks, hkv, d]
    qt = q.view(blocks, hkv, g, size, d)
    sink = torch.einsum("bhgtd,btshd->bhgts", qt, ks) / math.sqrt(d)
    sink = sink.masked_fill(~ok[:, None, None], -math.inf)
    top = torch.maximum(near.amax(-1), sink.amax(-1)) if sinks else near.amax(-1)
    near, sink = (near - top[..., None]).exp_(), (sink - top[..., None]).exp()
    o = (near.view(blocks, hkv, g * size, -1) @ v).view(blocks, hkv, g, size, d) + torch.einsum("bhgts,btshd->bhgtd", sink, vs)
    o = o / (near.sum(-1) + sink.sum(-1))[..., None]
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(pad, c["h_q"], d)[:t])


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        _own(s)
    elif op == "write":
        _plain_write(s)
    elif op == "read":
        _, _, _, block, row = _places(s)
        at = (block[:, None], torch.arange(s["case"]["h_kv"], device="cuda"), row[:, None])
        s["k_out"].copy_(_stored(s["pool_k"], s["scale_k"], at))
        s["v_out"].copy_(_stored(s["pool_v"], s["scale_v"], at))
    elif op == "chunk":
        _plain_chunk(s)
    else:
        _plain_window(s)
    if op == "window":
        return {"out": s["out"]}
    if op == "read":
        return {"k": s["k_out"], "v": s["v_out"]}
    r = {"pool_k": s["pool_k"], "pool_v": s["pool_v"]}
    if s["scale_k"] is not None:
        r.update(scale_k=s["scale_k"], scale_v=s["scale_v"])
    if op == "chunk":
        r["out"] = s["out"]
    return r


# ---------------------------------------------------------------------------------------------------------------
# the definition in 64 bits, question by question
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    lens, pre = s["host_lens"].tolist(), s["host_pre"].tolist()
    op, d, hq, hkv = case["op"], case["d"], case["h_q"], case["h_kv"]
    if op != "window" and case["op"] != "read" and s["scale_k"] is not None:
        scales = {"scale_k": s["scale_k"].double(), "scale_v": s["scale_v"].double()}
    elif op == "chunk":
        scales = {"scale_k": None, "scale_v": None}
    pairs, _ = _visible(case, np.array(lens), np.array(pre))
    if op in ("chunk", "window") and 4.0 * d * hq * pairs > 6e12:
        return None
    if op != "window":
        host_table = s["table"].cpu().numpy()
    outs, at = [], 0
    for i, (n, p) in enumerate(zip(lens, pre)):
        rows = slice(at, at + n)
        at += n
        if op == "window":
            k, v = s["k"][rows].double(), s["v"][rows].double()
        else:
            blocks = torch.from_numpy(host_table[i, :-(-(p + n) // PAGE)].astype(np.int64)).cuda()
            new = {"k": s["k"][rows].double(), "v": s["v"][rows].double()}
            full = {}
            for name in ("k", "v"):
                pool, scale = s["pool_" + name], s["scale_" + name]
                x = pool.view(torch.uint8)[blocks].view(torch.float8_e4m3fn).double() if scale is not None else pool[blocks].double()
                if scale is not None:
                    x = x * scale[blocks].double()[..., None]
                x = x.permute(0, 2, 1, 3).reshape(-1, hkv, d)[:p + n].clone()
                if op != "read":
                    y = new[name]
                    if scale is not None:
                        sc = y.abs().amax(-1) / E4M3_MAX
                        flat = torch.arange(p, p + n, device="cuda")
                        scales["scale_" + name][blocks[flat // PAGE], :, flat % PAGE] = sc
                        code = (y / sc[..., None]).float().clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).double()
                        y = torch.where(sc[..., None] == 0, torch.zeros_like(y), code * sc[..., None])
                    x[p:] = y
                full[name] = x
            k, v = full["k"], full["v"]
        if op == "read":
            outs.append((k[p:], v[p:]))
        elif op != "write":
            q = s["q"][rows].double().view(n, hkv, hq // hkv, d).permute(1, 2, 0, 3)
            o = torch.empty(hkv, hq // hkv, n, d, dtype=torch.float64, device="cuda")
            for a in range(0, n, 1024):  # rows a .. b of this question, over the positions that they can see
                b = min(n, a + 1024)
                lo = max(0, p + a - case["window"] + 1) if case["window"] else 0
                key = torch.cat([torch.arange(min(case["sinks"], lo)), torch.arange(lo, p + b)]).cuda()
                here = torch.arange(p + a, p + b, device="cuda")[:, None]
                seen = key <= here
                if case["window"]:
                    seen = seen & ((here - key < case["window"]) | (key < case["sinks"]))
                z = torch.einsum("hgtd,uhd->hgtu", q[:, :, a:b], k[key]) / math.sqrt(d)
                z = torch.where(seen, z, torch.full_like(z, -math.inf))
                o[:, :, a:b] = torch.einsum("hgtu,uhd->hgtd", torch.softmax(z, -1), v[key])
            outs.append(o.permute(2, 0, 1, 3).reshape(n, hq, d))
    if op == "read":
        return {"k": torch.cat([a for a, _ in outs]), "v": torch.cat([b for _, b in outs])}
    if op == "window":
        return {"out": torch.cat(outs)}
    r = {"pool_k": None, "pool_v": None}
    r.update({k: x for k, x in scales.items() if s["scale_k"] is not None})
    if op == "chunk":
        r["out"] = torch.cat(outs)
    return r
