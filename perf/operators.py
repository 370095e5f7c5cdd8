"""The operators of one verification round around the library's vocabulary-wide
calls, as cases to be measured:

  adjust  logits_adjust    penalties, biases and grammar masks on the logits of
                           drafted positions, before they are verified
  append  kv_append        the new tokens' keys and values rotated and appended
                           to a paged cache, their queries rotated
  attend  paged_attention  attention of the new tokens over the paged cache

``run`` computes them with elementary torch operations in 32 bits, or, where
``own`` is set, with this package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

# the benchmark batch's draft lengths
MIX = (2, 4, 8, 16)


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def _adjust(name, n, l_min, l_max, vocab, dtype, hist_min, hist_max, bias, masked, shape_seed, mix=False):
    return {"name": name, "op": "adjust", "n": n, "l_min": l_min, "l_max": l_max, "mix": mix, "vocab": vocab,
            "dtype": dtype, "hist_min": hist_min, "hist_max": hist_max, "bias": bias, "masked": masked,
            "shape_seed": shape_seed}


def _append(name, n, q_min, q_max, ctx_min, ctx_max, hq, hkv, d, rot, interleaved, page, dtype, shape_seed, mix=False):
    return {"name": name, "op": "append", "n": n, "q_min": q_min, "q_max": q_max, "mix": mix, "ctx_min": ctx_min,
            "ctx_max": ctx_max, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "interleaved": interleaved, "page": page,
            "dtype": dtype, "shape_seed": shape_seed}


def _attend(name, n, q_min, q_max, ctx_min, ctx_max, hq, hkv, d, page, causal, window, shape_seed, mix=False):
    return {"name": name, "op": "attend", "n": n, "q_min": q_min, "q_max": q_max, "mix": mix, "ctx_min": ctx_min,
            "ctx_max": ctx_max, "hq": hq, "hkv": hkv, "d": d, "page": page, "causal": causal, "window": window,
            "shape_seed": shape_seed}


def listed():
    return [
        # one request that decodes without a draft: one row, a short history, repetition penalties only
        _adjust("adjust one row", 1, 0, 0, 32000, "bf16", 64, 64, 0, 0, 1),
        # the benchmark's ragged batch with every feature on: histories of chats, biases, half of the requests
        # under a grammar
        _adjust("adjust mix", 256, 2, 16, 151936, "bf16", 128, 8192, 32, 2, 2, mix=True),
        # fp32 logits of a vocabulary whose rows are not 16-byte pitched, every request under a grammar
        _adjust("adjust fp32 odd", 32, 16, 16, 32003, "fp32", 1024, 1024, 300, 1, 3),
        # one token of one request
        _append("append one token", 1, 1, 1, 777, 777, 32, 8, 128, 128, False, 16, "bf16", 4),
        # the benchmark's ragged batch: the drafted tokens and the last emitted one of every request
        _append("append mix", 256, 3, 17, 64, 900, 32, 8, 128, 128, False, 64, "bf16", 5, mix=True),
        # prompts in chunks, a drafter's small heads, a partial interleaved rotation, one key head per query head
        _append("append prompts", 5, 1500, 4096, 0, 1000, 16, 16, 64, 32, True, 32, "bf16", 6),
        # one token of one request: latency
        _attend("attend one token", 1, 1, 1, 777, 777, 32, 8, 128, 16, True, 0, 7),
        # plain decoding: one token each, long ragged contexts
        _attend("attend decode", 64, 1, 1, 1000, 16000, 32, 8, 128, 64, True, 0, 8),
        # the benchmark's ragged batch of verified blocks
        _attend("attend mix", 256, 3, 17, 512, 8192, 32, 8, 128, 32, True, 0, 9, mix=True),
        # one request's block over a long document: the work is split over the keys
        _attend("attend long", 1, 17, 17, 131000, 131000, 32, 8, 128, 64, True, 0, 10),
        # chunks of two prompts over what is cached of them: bound by the tensor cores
        _attend("attend prompts", 2, 2048, 2048, 8192, 8192, 32, 8, 128, 128, True, 0, 11),
        # a diffusion drafter's block: every position sees the whole block; small heads, no sharing
        _attend("attend draft block", 128, 16, 16, 200, 2000, 16, 16, 64, 32, False, 0, 12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("adjust", "append", "attend"))
    seed = rng.randrange(1 << 20)
    if op == "adjust":
        vocab = _log(rng, 2000, 152000) | 1  # rows that are not 16-byte pitched
        if rng.random() < 0.6:
            vocab = vocab // 16 * 16 + 8  # and rows that are
        n = _log(rng, 1, 256)
        l_max = rng.choice((0, 1, 3, 8, 16))
        hist = _log(rng, 16, 8192)
        c = _adjust("", n, min(l_max, rng.choice((0, 1, l_max))), l_max, vocab, rng.choice(("bf16", "bf16", "fp32")),
                    rng.choice((0, hist // 4)), hist | 1, rng.choice((0, 0, 7, 32, 300)), rng.choice((0, 1, 2)), seed)
        while work(c)["bytes"] > 1.2e9:
            c["n"] = max(1, c["n"] // 2)
    elif op == "append":
        hkv = rng.choice((1, 2, 4, 8, 16))
        d = rng.choice((64, 128))
        q_max = _log(rng, 1, 4095) | 1
        n = min(_log(rng, 1, 256), max(1, 16384 // q_max))
        c = _append("", n, rng.choice((1, q_max // 2 + 1, q_max)), q_max, 0, rng.choice((0, 100, 900)),
                    hkv * rng.choice((1, 2, 4, 5, 7, 8)), hkv, d, rng.choice((d, d, d // 2)), rng.random() < 0.3,
                    rng.choice((16, 32, 64, 128)), rng.choice(("bf16", "bf16", "fp32")), seed)
        while work(c)["bytes"] > 3e8:
            c["n"] = max(1, c["n"] // 2)
            if c["n"] == 1:
                c["q_max"] = max(1, c["q_max"] // 2)
                c["q_min"] = min(c["q_min"], c["q_max"])
    else:
        hkv = rng.choice((1, 2, 4, 8, 16))
        d = rng.choice((64, 128))
        q_max = _log(rng, 1, 1500) | 1
        ctx = _log(rng, 16, 60000) | 1
        n = _log(rng, 1, 256)
        c = _attend("", n, rng.choice((1, q_max // 2 + 1, q_max)), q_max, rng.choice((0, ctx // 8, ctx)), ctx,
                    hkv * rng.choice((1, 2, 4, 5, 7, 8)), hkv, d, rng.choice((16, 32, 64, 128)), rng.random() < 0.8, 0, seed)
        if c["causal"] and rng.random() < 0.2:
            c["window"] = _log(rng, 16, 4096) | 1
        while True:
            w = work(c)
            padded = c["n"] * c["hq"] * c["q_max"] * (c["ctx_max"] + c["q_max"])
            if w["bytes"] < 3e9 and w["flops"] < 4e11 and padded < 1.5e9:
                break
            if c["n"] > 1:
                c["n"] //= 2
            elif c["ctx_max"] > 4000:
                c["ctx_max"] //= 2
                c["ctx_min"] = min(c["ctx_min"], c["ctx_max"])
            else:
                c["q_max"] //= 2
                c["q_min"] = min(c["q_min"], c["q_max"])
    del c["name"]
    return c


def _lengths(case):
    """New tokens (draft positions) and cached tokens (history) of each request, from the case alone."""
    rng = random.Random(case["shape_seed"])
    adjust = case["op"] == "adjust"
    lo, hi = (case["l_min"], case["l_max"]) if adjust else (case["q_min"], case["q_max"])
    c_lo, c_hi = (case["hist_min"], case["hist_max"]) if adjust else (case["ctx_min"], case["ctx_max"])
    new, old = [], []
    for _ in range(case["n"]):
        if case["mix"]:
            new.append(rng.choice(MIX) + (0 if adjust else 1))
        else:
            new.append(lo if lo == hi else min(hi, rng.randint(lo, hi) | 1))
        old.append(c_lo if c_lo == c_hi else int(math.exp(rng.uniform(math.log(c_lo + 1), math.log(c_hi + 1))) - 0.5))
    return new, old


def _visible(case, q, kv):
    """Keys that q new tokens at the end of kv tokens see, summed over the tokens."""
    if not case["causal"]:
        return q * kv
    at = np.arange(kv - q, kv, dtype=np.int64)
    lo = np.maximum(0, at + 1 - case["window"]) if case["window"] else 0
    return int((at + 1 - lo).sum())


def work(case):
    new, old = _lengths(case)
    es = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if case["op"] == "adjust":
        rows, v = sum(new) + case["n"], case["vocab"]
        under = sum(l + 1 for i, l in enumerate(new) if case["masked"] and i % case["masked"] == 0)
        b = 2 * rows * v * es + under * ((v + 31) // 32) * 4 + 4 * (sum(old) + sum(new)) + 8 * case["bias"] * case["n"]
        return {"bytes": float(b), "flops": float(rows * v)}
    t = sum(new)
    if case["op"] == "append":
        moved = 2 * t * (case["hq"] + 2 * case["hkv"]) * case["d"] * es + t * case["rot"] * 4
        return {"bytes": float(moved), "flops": float(3 * t * (case["hq"] + case["hkv"]) * case["rot"])}
    seen = keys = 0
    for q, c in zip(new, old):
        seen += _visible(case, q, q + c)
        keys += q + (min(c, case["window"] - 1) if case["window"] else c)
    b = 2 * t * case["hq"] * case["d"] * 2 + 4 * t * case["hq"] + 2 * keys * case["hkv"] * case["d"] * 2
    return {"bytes": float(b), "flops": float(4 * case["d"] * case["hq"] * seen)}


# ---------------------------------------------------------------------------
# what a program has in hand before the call
# ---------------------------------------------------------------------------
def _csr(lens):
    return torch.tensor([0] + list(np.cumsum(lens, dtype=np.int64)), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    new, old = _lengths(case)
    dev, n = "cuda", case["n"]
    dt = torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32

    def randint(hi, shape):
        return torch.randint(0, hi, shape, generator=g, device=dev, dtype=torch.int32)

    s = {"case": case}
    if case["op"] == "adjust":
        v, drafts = case["vocab"], sum(new)
        rows = drafts + n
        s["logits"] = torch.empty(rows, v, dtype=dt, device=dev).normal_(0, 3, generator=g)
        # text repeats itself: tokens from a few hundred frequent ones and from the whole vocabulary
        few = randint(min(v, 500), (sum(old),))
        s["history"] = torch.where(torch.rand(sum(old), generator=g, device=dev) < 0.5, few, randint(v, (sum(old),)))
        s["cu_history"] = _csr(old)
        s["prompt_len"] = torch.tensor([c // 2 for c in old], dtype=torch.int32, device=dev)
        s["cu_draft"] = _csr(new)
        s["drafts"] = drafts
        s["draft_tokens"] = torch.where(torch.rand(drafts, generator=g, device=dev) < 0.5,
                                        randint(min(v, 500), (drafts,)), randint(v, (drafts,)))
        s["repetition"] = 1 + 0.3 * torch.rand(n, generator=g, device=dev)
        s["frequency"] = 0.5 * torch.rand(n, generator=g, device=dev)
        s["presence"] = 0.5 * torch.rand(n, generator=g, device=dev)
        s["bias_tokens"] = s["bias_values"] = s["cu_bias"] = s["mask"] = s["mask_row"] = None
        if nb := min(case["bias"], v):
            # different tokens within a request: v // nb apart
            first = randint(v, (n, 1))
            step = torch.arange(nb, device=dev, dtype=torch.int32) * (v // nb)
            s["bias_tokens"] = ((first + step) % v).to(torch.int32).reshape(-1)
            b = 4 * torch.randn(n * nb, generator=g, device=dev)
            s["bias_values"] = torch.where(b < -6, -torch.inf, b)  # a few banned tokens
            s["cu_bias"] = _csr([nb] * n)
        if case["masked"]:
            under = [l + 1 if i % case["masked"] == 0 else 0 for i, l in enumerate(new)]
            w = (v + 31) // 32
            mask = torch.randint(-2**31, 2**31, (sum(under), w), generator=g, device=dev, dtype=torch.int64)
            more = torch.randint(-2**31, 2**31, (sum(under), w), generator=g, device=dev, dtype=torch.int64)
            narrow = torch.rand(sum(under), 1, generator=g, device=dev)
            # a grammar's states: inside a string nearly every token is allowed, at a keyword a few
            some = (torch.rand(sum(under), w, generator=g, device=dev) < 0.01) * (mask & more)
            s["mask"] = torch.where(narrow < 0.5, some, torch.where(narrow < 0.8, mask | more, -1)).to(torch.int32)
            at, rows_of = 0, []
            for u, l in zip(under, new):
                rows_of += list(range(at, at + u)) if u else [-1] * (l + 1)
                at += u
            s["mask_row"] = torch.tensor(rows_of, dtype=torch.int32, device=dev)
        s["out"] = torch.empty_like(s["logits"])
        return s

    t, hq, hkv, d, page = sum(new), case["hq"], case["hkv"], case["d"], case["page"]
    pages = [(q + c + page - 1) // page for q, c in zip(new, old)]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((n, max(pages)), -1, dtype=torch.int32, device=dev)
    at = torch.tensor([0] + list(np.cumsum(pages))[:-1], device=dev)
    col = torch.arange(max(pages), device=dev)
    used = col[None] < torch.tensor(pages, device=dev)[:, None]
    table = torch.where(used, order[(at[:, None] + col[None]).clamp(max=n_pages - 1)], table)
    s["block_table"] = table
    s["cu_new"] = _csr(new)
    s["kv_len"] = torch.tensor([q + c for q, c in zip(new, old)], dtype=torch.int32, device=dev)
    s["max_new"], s["max_kv"] = max(new), max(q + c for q, c in zip(new, old))
    s["k_cache"] = torch.empty(n_pages, hkv, page, d, dtype=dt, device=dev).normal_(0, 1, generator=g)
    s["v_cache"] = torch.empty(n_pages, hkv, page, d, dtype=dt, device=dev).normal_(0, 1, generator=g)
    if case["op"] == "append":
        qkv = torch.empty(t, (hq + 2 * hkv) * d, dtype=dt, device=dev).normal_(0, 1, generator=g)
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
        inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev) / case["rot"])
        # a table from another start for every seed, as a program with a scaled rotation would keep
        angle = torch.arange(s["max_kv"], dtype=torch.float64, device=dev)[:, None] * inv * (1 + (seed % 97) / 100)
        s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), 1).to(torch.float32)
        s["q_out"] = torch.empty(t, hq, d, dtype=dt, device=dev)
    else:
        s["q"] = torch.empty(t, hq, d, dtype=dt, device=dev).normal_(0, 1.5, generator=g)
        s["scale"] = 1 / math.sqrt(d)
        s["out"] = torch.empty(t, hq, d, dtype=dt, device=dev)
        s["lse"] = torch.empty(t, hq, dtype=torch.float32, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"adjust": _own_adjust, "append": _own_append, "attend": _own_attend}[op](s)
    return {"adjust": _plain_adjust, "append": _plain_append, "attend": _plain_attend}[op](s)


def _own_adjust(s):
    import serving_vocab_wide_gb300 as svw
    return svw.logits_adjust(s["logits"], s["cu_draft"], s["draft_tokens"], history=s["history"],
                             cu_history=s["cu_history"], prompt_len=s["prompt_len"], repetition=s["repetition"],
                             frequency=s["frequency"], presence=s["presence"], bias_tokens=s["bias_tokens"],
                             bias_values=s["bias_values"], cu_bias=s["cu_bias"], mask=s["mask"],
                             mask_row=s["mask_row"], has_bonus=True, total_draft_rows=s["drafts"], out=s["out"])


def _own_append(s):
    import serving_vocab_wide_gb300 as svw
    q = svw.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_new"], s["kv_len"],
                      cos_sin=s["cos_sin"], interleaved=s["case"]["interleaved"], q=s["q"], q_out=s["q_out"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    import serving_vocab_wide_gb300 as svw
    out, lse = svw.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_new"], s["kv_len"],
                                   scale=s["scale"], causal=s["case"]["causal"], window=s["case"]["window"],
                                   out=s["out"], lse=s["lse"])
    return {"out": out, "lse": lse}


def _owner(cu, count):
    """The request of each of `count` packed entries, and its place in the request."""
    at = torch.arange(count, device=cu.device, dtype=torch.int32)
    who = torch.searchsorted(cu[1:], at, right=True)
    return who, at - cu[who]


def _plain_adjust(s):
    x = s["logits"].float()
    rows, v = x.shape
    n, dev = s["cu_draft"].numel() - 1, x.device
    cu_rows = s["cu_draft"] + torch.arange(n + 1, device=dev, dtype=torch.int32)
    who, j = _owner(cu_rows, rows)
    hw, hj = _owner(s["cu_history"], s["history"].numel())
    in_prompt = hj < s["prompt_len"][hw]
    where = hw * v + s["history"]
    prompt = torch.zeros(n * v, dtype=torch.int32, device=dev).index_put_((where,), in_prompt.int(), accumulate=True)
    count = torch.zeros(n * v, dtype=torch.int32, device=dev).index_put_((where,), (~in_prompt).int(), accumulate=True)
    prompt, count = prompt.view(n, v)[who], count.view(n, v)[who]
    longest = s["case"]["l_max"]
    if s["drafts"]:
        back = torch.arange(longest, device=dev)
        before = back[None] < j[:, None]  # row j has seen the drafted tokens before it
        tok = s["draft_tokens"][(s["cu_draft"][who][:, None] + back[None]).clamp(max=s["drafts"] - 1)]
        count.scatter_add_(1, torch.where(before, tok, 0).long(), before.int())
    seen = (prompt > 0) | (count > 0)
    rep = s["repetition"][who][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][who][:, None] * count - s["presence"][who][:, None] * (count > 0)
    if s["cu_bias"] is not None:
        bw, _ = _owner(s["cu_bias"], s["bias_tokens"].numel())
        bias = torch.zeros(n * v, device=dev).index_put_((bw * v + s["bias_tokens"],), s["bias_values"])
        x = x + bias.view(n, v)[who]
    if s["mask"] is not None:
        tok = torch.arange(v, device=dev)
        words = s["mask"][s["mask_row"].clamp(min=0)]
        allowed = (words[:, tok >> 5] >> (tok & 31).int()[None]) & 1
        x = torch.where((allowed == 1) | (s["mask_row"] < 0)[:, None], x, -torch.inf)
    s["out"].copy_(x)
    return s["out"]


def _rotated(x, cs, rot, interleaved):
    c, sn = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * c - b * sn, b * c + a * sn
    y = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_append(s):
    c = s["case"]
    t, page = s["k"].shape[0], c["page"]
    who, j = _owner(s["cu_new"], t)
    new = s["cu_new"][1:] - s["cu_new"][:-1]
    at = s["kv_len"][who] - new[who] + j
    cs = s["cos_sin"][at]
    slot, row = s["block_table"][who, at // page].long(), (at % page).long()
    dt = s["k"].dtype
    s["k_cache"][slot, :, row] = _rotated(s["k"].float(), cs, c["rot"], c["interleaved"]).to(dt)
    s["v_cache"][slot, :, row] = s["v"]
    s["q_out"].copy_(_rotated(s["q"].float(), cs, c["rot"], c["interleaved"]))
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    c = s["case"]
    n, t, hq, hkv, d = c["n"], s["q"].shape[0], c["hq"], c["hkv"], c["d"]
    mq, page, dev = s["max_new"], c["page"], s["q"].device
    table = s["block_table"].clamp(min=0)
    mk = table.shape[1] * page
    k = s["k_cache"][table].float().permute(0, 2, 1, 3, 4).reshape(n, hkv, mk, d)
    key = torch.arange(mk, device=dev)
    real = key[None] < s["kv_len"][:, None]
    new = s["cu_new"][1:] - s["cu_new"][:-1]
    tok = torch.arange(mq, device=dev)
    at = (s["cu_new"][:-1, None] + tok[None]).clamp(max=t - 1)
    q = s["q"][at].float().view(n, mq, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, -1, d)
    x = torch.matmul(q, k.transpose(2, 3)).view(n, hkv, mq, hq // hkv, mk)
    x *= s["scale"]
    pos = s["kv_len"][:, None] - new[:, None] + tok[None]
    ok = real[:, None, :].expand(n, mq, mk)
    if c["causal"]:
        ok = ok & (key[None, None] <= pos[..., None])
        if c["window"]:
            ok = ok & (key[None, None] > pos[..., None] - c["window"])
    x.masked_fill_(~ok[:, None, :, None], -torch.inf)
    m = x.max(-1, keepdim=True).values
    m = torch.where(m == -torch.inf, 0.0, m)  # a row without keys
    x = torch.exp(x.sub_(m))
    total = x.sum(-1, keepdim=True)
    v = s["v_cache"][table].float().permute(0, 2, 1, 3, 4).reshape(n, hkv, mk, d)
    v = torch.where(real[:, None, :, None], v, 0.0)
    y = torch.matmul(x.view(n, hkv, -1, mk), v).view(n, hkv, mq, hq // hkv, d)
    y = torch.where(total > 0, y / total, 0.0)
    lse = (m + torch.log(total))[..., 0]
    who, j = _owner(s["cu_new"], t)
    s["out"].copy_(y.permute(0, 2, 1, 3, 4)[who, j].reshape(t, hq, d))
    s["lse"].copy_(lse.permute(0, 2, 1, 3)[who, j].reshape(t, hq))
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, request by request
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"adjust": _exact_adjust, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)


def _exact_adjust(s):
    v = s["logits"].shape[1]
    out = s["logits"].double()
    cu, cuh = s["cu_draft"].tolist(), s["cu_history"].tolist()
    rep, freq, pres = s["repetition"].tolist(), s["frequency"].tolist(), s["presence"].tolist()
    bits = torch.arange(32, device=out.device, dtype=torch.int32)
    for i in range(len(cu) - 1):
        hist = s["history"][cuh[i]:cuh[i + 1]].long()
        p = int(s["prompt_len"][i])
        told = torch.bincount(hist[:p], minlength=v) > 0
        said = torch.bincount(hist[p:], minlength=v).double()
        for j in range(cu[i + 1] - cu[i] + 1):
            x = out[cu[i] + i + j]
            if j:
                said[s["draft_tokens"][cu[i] + j - 1].long()] += 1
            old = told | (said > 0)
            y = torch.where(x > 0, x / rep[i], x * rep[i])
            y = torch.where(old, y, x) - freq[i] * said - pres[i] * (said > 0).double()
            if s["cu_bias"] is not None:
                b0, b1 = int(s["cu_bias"][i]), int(s["cu_bias"][i + 1])
                y[s["bias_tokens"][b0:b1].long()] += s["bias_values"][b0:b1].double()
            if s["mask"] is not None and (r := int(s["mask_row"][cu[i] + i + j])) >= 0:
                allowed = ((s["mask"][r][:, None] >> bits) & 1).reshape(-1)[:v] == 1
                y[~allowed] = -math.inf
            out[cu[i] + i + j] = y
    return out


def _exact_append(s):
    c = s["case"]
    rot, page = c["rot"], c["page"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    q = s["q"].double().clone()
    cu, kv = s["cu_new"].tolist(), s["kv_len"].tolist()
    first = torch.arange(0, rot, 2) if c["interleaved"] else torch.arange(rot // 2)
    second = first + (1 if c["interleaved"] else rot // 2)
    first, second = first.cuda(), second.cuda()
    for i in range(c["n"]):
        at = torch.arange(kv[i] - (cu[i + 1] - cu[i]), kv[i], device="cuda")
        z = torch.complex(*s["cos_sin"][at].double().chunk(2, 1))[:, None]
        k = s["k"][cu[i]:cu[i + 1]].double()
        for x in (k, q[cu[i]:cu[i + 1]]):
            y = torch.complex(x[..., first], x[..., second]) * z
            x[..., first], x[..., second] = y.real, y.imag
        slot = s["block_table"][i][at // page].long()
        kc[slot, :, at % page] = k
        vc[slot, :, at % page] = s["v"][cu[i]:cu[i + 1]].double()
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _exact_attend(s):
    c = s["case"]
    g = c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    cu, kv = s["cu_new"].tolist(), s["kv_len"].tolist()
    for i in range(c["n"]):
        a, b = cu[i], cu[i + 1]
        slots = s["block_table"][i][:(kv[i] + c["page"] - 1) // c["page"]].long()
        k = s["k_cache"][slots].double().transpose(1, 2).reshape(-1, c["hkv"], c["d"])[:kv[i]]
        v = s["v_cache"][slots].double().transpose(1, 2).reshape(-1, c["hkv"], c["d"])[:kv[i]]
        at = torch.arange(kv[i] - (b - a), kv[i], device="cuda")[:, None]
        key = torch.arange(kv[i], device="cuda")[None]
        hidden = torch.zeros(b - a, kv[i], dtype=torch.bool, device="cuda")
        if c["causal"]:
            hidden = key > at
            if c["window"]:
                hidden |= key <= at - c["window"]
        for h in range(c["hq"]):
            x = (s["q"][a:b, h].double() @ k[:, h // g].T) * s["scale"]
            x = x.masked_fill(hidden, -math.inf)
            lse[a:b, h] = torch.logsumexp(x, 1)
            out[a:b, h] = torch.exp(x - lse[a:b, h, None]) @ v[:, h // g]
    return {"out": out, "lse": lse}
