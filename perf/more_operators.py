"""A paged key-value cache of 8 bits, as cases to be measured: what writes it,
what attends over it and what reads it back.

  append  kv_append_norm       the new tokens' keys and queries normed per head
                               and rotated, keys and values written in e4m3
                               with a scale for each head
  attend  paged_attention_fp8  attention of the new tokens over that cache
  gather  kv_gather            cached tokens read back, packed

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
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def _append(name, n, q_min, q_max, ctx_min, ctx_max, hq, hkv, d, rot, interleaved, normed, page, dtype, cache,
            shape_seed, mix=False):
    return {"name": name, "op": "append", "n": n, "q_min": q_min, "q_max": q_max, "mix": mix, "ctx_min": ctx_min,
            "ctx_max": ctx_max, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "interleaved": interleaved,
            "normed": normed, "page": page, "dtype": dtype, "cache": cache, "shape_seed": shape_seed}


def _attend(name, n, q_min, q_max, ctx_min, ctx_max, hq, hkv, d, page, causal, window, shape_seed, mix=False):
    return {"name": name, "op": "attend", "n": n, "q_min": q_min, "q_max": q_max, "mix": mix, "ctx_min": ctx_min,
            "ctx_max": ctx_max, "hq": hq, "hkv": hkv, "d": d, "page": page, "causal": causal, "window": window,
            "cache": "e4m3", "shape_seed": shape_seed}


def _gather(name, n, len_min, len_max, skip, hkv, d, page, cache, out, shape_seed):
    """From cached token `skip` of each request on, len_min to len_max of them."""
    return {"name": name, "op": "gather", "n": n, "q_min": len_min, "q_max": len_max, "mix": False, "ctx_min": skip,
            "ctx_max": skip, "hkv": hkv, "d": d, "page": page, "cache": cache, "out": out, "shape_seed": shape_seed}


def listed():
    return [
        # one token of one request: latency
        _append("append one token", 1, 1, 1, 777, 777, 32, 8, 128, 128, False, True, 16, "bf16", "e4m3", 1),
        # the benchmark's ragged batch: the drafted tokens and the last emitted one of every request
        _append("append mix", 256, 3, 17, 64, 900, 32, 8, 128, 128, False, True, 64, "bf16", "e4m3", 2, mix=True),
        # prompts in chunks: small heads, a partial interleaved rotation, one key head per query head, no norms
        _append("append prompts", 5, 1500, 4096, 0, 1000, 16, 16, 64, 32, True, False, 32, "bf16", "e4m3", 3),
        # a model with norms whose cache stays in bf16
        _append("append bf16 cache", 100, 1, 33, 64, 900, 40, 8, 128, 128, False, True, 16, "bf16", "bf16", 4),
        # one request's cache handed on
        _gather("gather one", 1, 777, 777, 0, 8, 128, 16, "e4m3", "bf16", 5),
        # the ends of many requests' caches, as a drafter takes them
        _gather("gather many", 64, 1000, 9000, 333, 8, 128, 64, "e4m3", "bf16", 6),
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
    op = rng.choice(("append", "attend", "attend", "gather"))
    seed = rng.randrange(1 << 20)
    hkv = rng.choice((1, 2, 4, 8, 16))
    if op == "append":
        d = rng.choice((64, 96, 128, 128, 256))
        q_max = _log(rng, 1, 4095) | 1
        n = min(_log(rng, 1, 256), max(1, 16384 // q_max))
        c = _append("", n, rng.choice((1, q_max // 2 + 1, q_max)), q_max, 0, rng.choice((0, 100, 900)),
                    hkv * rng.choice((1, 2, 4, 5, 7, 8)), hkv, d, rng.choice((d, d, d // 2)), rng.random() < 0.3,
                    rng.random() < 0.7, rng.choice((16, 32, 64, 128)), rng.choice(("bf16", "bf16", "fp32")),
                    "e4m3", seed)
        if rng.random() < 0.25:
            c["cache"] = c["dtype"]
        while work(c)["bytes"] > 3e8:
            c["n"] = max(1, c["n"] // 2)
            if c["n"] == 1:
                c["q_max"] = max(1, c["q_max"] // 2)
                c["q_min"] = min(c["q_min"], c["q_max"])
    elif op == "gather":
        q_max = _log(rng, 1, 20000) | 1
        n = _log(rng, 1, 256)
        c = _gather("", n, rng.choice((1, q_max // 2 + 1, q_max)), q_max, rng.choice((0, 1, 50, 1000)), hkv,
                    rng.choice((64, 96, 128, 128, 256)), rng.choice((16, 32, 64, 128)),
                    rng.choice(("e4m3", "e4m3", "bf16")), rng.choice(("bf16", "bf16", "fp32")), seed)
        while work(c)["bytes"] > 1.2e9:
            if c["n"] > 1:
                c["n"] //= 2
            else:
                c["q_max"] //= 2
                c["q_min"] = min(c["q_min"], c["q_max"])
    else:
        d = rng.choice((64, 128))
        q_max = _log(rng, 1, 1500) | 1
        ctx = _log(rng, 16, 60000) | 1
        n = _log(rng, 1, 256)
        c = _attend("", n, rng.choice((1, q_max // 2 + 1, q_max)), q_max, rng.choice((0, ctx // 8, ctx)), ctx,
                    hkv * rng.choice((1, 2, 4, 5, 7, 8)), hkv, d, rng.choice((16, 32, 64, 128)), rng.random() < 0.8, 0,
                    seed)
        if c["causal"] and rng.random() < 0.2:
            c["window"] = _log(rng, 16, 4096) | 1
        while True:
            w = work(c)
            padded = c["n"] * c["hq"] * c["q_max"] * (c["ctx_max"] + c["q_max"])
            if w["bytes"] < 1.5e9 and w["flops"] < 4e11 and padded < 1.5e9:
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
    """New tokens (tokens read back) and the cached ones before them of each request, from the case alone."""
    rng = random.Random(case["shape_seed"])
    lo, hi, c_lo, c_hi = case["q_min"], case["q_max"], case["ctx_min"], case["ctx_max"]
    new, old = [], []
    for _ in range(case["n"]):
        if case["mix"]:
            new.append(rng.choice(MIX) + 1)
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


SIZE = {"fp32": 4, "bf16": 2, "e4m3": 1}


def work(case):
    new, old = _lengths(case)
    t, hkv, d, es = sum(new), case["hkv"], case["d"], SIZE[case["cache"]]
    if case["op"] == "append":
        read = t * (case["hq"] + 2 * hkv) * d * SIZE[case["dtype"]] + t * case["rot"] * 4
        written = t * case["hq"] * d * SIZE[case["dtype"]] + 2 * t * hkv * d * es
        each = 3 * case["rot"] + (4 * d if case["normed"] else 0)
        return {"bytes": float(read + written), "flops": float(t * (case["hq"] + hkv) * each + 2 * t * hkv * d)}
    if case["op"] == "gather":
        return {"bytes": float(2 * t * hkv * d * (es + SIZE[case["out"]])), "flops": float(2 * t * hkv * d)}
    seen = keys = 0
    for q, c in zip(new, old):
        seen += _visible(case, q, q + c)
        keys += q + (min(c, case["window"] - 1) if case["window"] else c)
    b = 2 * t * case["hq"] * d * 2 + 4 * t * case["hq"] + 2 * keys * hkv * d * es
    return {"bytes": float(b), "flops": float(4 * d * case["hq"] * seen)}


# ---------------------------------------------------------------------------
# what a program has in hand before the call
# ---------------------------------------------------------------------------
DTYPE = {"fp32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def _csr(lens):
    return torch.tensor([0] + list(np.cumsum(lens, dtype=np.int64)), dtype=torch.int32, device="cuda")


def _cached(shape, scale, dtype, g):
    """A cache that holds unit normal values, in units of each head's scale where it is of 8 bits."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    if dtype == torch.float8_e4m3fn:
        x = (x / scale.to(torch.bfloat16)[None, :, None, None]).clamp_(-E4M3_MAX, E4M3_MAX)
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    new, old = _lengths(case)
    dev, n, hkv, d, page = "cuda", case["n"], case["hkv"], case["d"], case["page"]
    t = sum(new)
    s = {"case": case}
    pages = [(q + c + page - 1) // page for q, c in zip(new, old)]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((n, max(pages)), -1, dtype=torch.int32, device=dev)
    at = torch.tensor([0] + list(np.cumsum(pages))[:-1], device=dev)
    col = torch.arange(max(pages), device=dev)
    used = col[None] < torch.tensor(pages, device=dev)[:, None]
    s["block_table"] = torch.where(used, order[(at[:, None] + col[None]).clamp(max=n_pages - 1)], table)
    s["cu_new"] = _csr(new)
    s["kv_len"] = torch.tensor([q + c for q, c in zip(new, old)], dtype=torch.int32, device=dev)
    s["max_new"], s["max_kv"] = max(new), max(q + c for q, c in zip(new, old))
    # a head's largest value, as found beforehand, at the end of e4m3's range
    most = 5 + 3 * torch.rand(2, hkv, generator=g, device=dev)
    if case["op"] == "append" and case["normed"]:
        most[0] *= 1.5  # the weights of the norm
    s["k_scale"] = s["v_scale"] = None
    if case["cache"] == "e4m3":
        s["k_scale"], s["v_scale"] = (most / E4M3_MAX).contiguous()
    shape, ct = (n_pages, hkv, page, d), DTYPE[case["cache"]]
    s["k_cache"] = _cached(shape, s["k_scale"], ct, g)
    s["v_cache"] = _cached(shape, s["v_scale"], ct, g)
    if case["op"] == "append":
        hq, dt, rot = case["hq"], DTYPE[case["dtype"]], case["rot"]
        qkv = torch.empty(t, (hq + 2 * hkv) * d, dtype=torch.float32, device=dev).normal_(0, 1, generator=g)
        qkv *= 1 + torch.rand((hq + 2 * hkv) * d, generator=g, device=dev) * (1 if case["normed"] else 0)
        qkv = qkv.to(dt)
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
        s["q_weight"] = s["k_weight"] = None
        if case["normed"]:
            s["q_weight"], s["k_weight"] = (0.7 + 0.8 * torch.rand(2, d, generator=g, device=dev)).contiguous()
        inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
        # a table from another start for every seed, as a program with a scaled rotation would keep
        angle = torch.arange(s["max_kv"], dtype=torch.float64, device=dev)[:, None] * inv * (1 + (seed % 97) / 100)
        s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), 1).to(torch.float32)
        s["q_out"] = torch.empty(t, hq, d, dtype=dt, device=dev)
    elif case["op"] == "gather":
        s["first"] = torch.tensor(old, dtype=torch.int32, device=dev)
        s["k_out"], s["v_out"] = torch.empty(2, t, hkv, d, dtype=DTYPE[case["out"]], device=dev)
    else:
        hq = case["hq"]
        s["q"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device=dev).normal_(0, 1.5, generator=g)
        s["scale"] = 1 / math.sqrt(d)
        s["out"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(t, hq, dtype=torch.float32, device=dev)
    return s


EPS = 1e-6


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "gather": _own_gather}[op](s)
    return {"append": _plain_append, "attend": _plain_attend, "gather": _plain_gather}[op](s)


def _own_append(s):
    import serving_vocab_wide_gb300 as svw
    q = svw.kv_append_norm(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_new"], s["kv_len"],
                           k_weight=s["k_weight"], q_weight=s["q_weight"], eps=EPS, k_scale=s["k_scale"],
                           v_scale=s["v_scale"], cos_sin=s["cos_sin"], interleaved=s["case"]["interleaved"], q=s["q"],
                           q_out=s["q_out"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    import serving_vocab_wide_gb300 as svw
    out, lse = svw.paged_attention_fp8(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_new"], s["kv_len"],
                                       k_scale=s["k_scale"], v_scale=s["v_scale"], scale=s["scale"],
                                       causal=s["case"]["causal"], window=s["case"]["window"], out=s["out"],
                                       lse=s["lse"])
    return {"out": out, "lse": lse}


def _own_gather(s):
    import serving_vocab_wide_gb300 as svw
    k, v = svw.kv_gather(s["k_cache"], s["v_cache"], s["block_table"], s["cu_new"], first=s["first"],
                         k_scale=s["k_scale"], v_scale=s["v_scale"], k_out=s["k_out"], v_out=s["v_out"])
    return {"k": k, "v": v}


def _owner(cu, count):
    """The request of each of `count` packed entries, and its place in the request."""
    at = torch.arange(count, device=cu.device, dtype=torch.int32)
    who = torch.searchsorted(cu[1:], at, right=True)
    return who, at - cu[who]


def _normed(x, weight):
    x = x.float()
    return x if weight is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


def _rotated(x, cs, rot, interleaved):
    c, sn = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * c - b * sn, b * c + a * sn
    y = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _stored(x, scale, dtype):
    """Values as they are kept, heads second to last; codes are moved as bytes."""
    if scale is None:
        return x.to(dtype)
    return (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(dtype).view(torch.uint8)


def _bytes(cache):
    return cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache


def _plain_append(s):
    c = s["case"]
    t, page = s["k"].shape[0], c["page"]
    who, j = _owner(s["cu_new"], t)
    new = s["cu_new"][1:] - s["cu_new"][:-1]
    at = s["kv_len"][who] - new[who] + j
    cs = s["cos_sin"][at]
    slot, row = s["block_table"][who, at // page].long(), (at % page).long()
    k = _rotated(_normed(s["k"], s["k_weight"]), cs, c["rot"], c["interleaved"])
    _bytes(s["k_cache"])[slot, :, row] = _stored(k, s["k_scale"], s["k_cache"].dtype)
    _bytes(s["v_cache"])[slot, :, row] = _stored(s["v"].float(), s["v_scale"], s["v_cache"].dtype)
    s["q_out"].copy_(_rotated(_normed(s["q"], s["q_weight"]), cs, c["rot"], c["interleaved"]))
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _read(cache, scale, slot, row):
    x = _bytes(cache)[slot, :, row].contiguous().view(cache.dtype).float()
    return x if scale is None else x * scale[:, None]


def _plain_gather(s):
    page = s["case"]["page"]
    who, j = _owner(s["cu_new"], s["k_out"].shape[0])
    at = s["first"][who] + j
    slot, row = s["block_table"][who, at // page].long(), (at % page).long()
    s["k_out"].copy_(_read(s["k_cache"], s["k_scale"], slot, row))
    s["v_out"].copy_(_read(s["v_cache"], s["v_scale"], slot, row))
    return {"k": s["k_out"], "v": s["v_out"]}


def _pages(cache, scale, table, shape):
    x = _bytes(cache)[table].view(cache.dtype).float()
    return (x * scale[:, None, None]).permute(0, 2, 1, 3, 4).reshape(shape)


def _plain_attend(s):
    c = s["case"]
    n, t, hq, hkv, d = c["n"], s["q"].shape[0], c["hq"], c["hkv"], c["d"]
    mq, page, dev = s["max_new"], c["page"], s["q"].device
    table = s["block_table"].clamp(min=0)
    mk = table.shape[1] * page
    k = _pages(s["k_cache"], s["k_scale"], table, (n, hkv, mk, d))
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
    del k
    v = _pages(s["v_cache"], s["v_scale"], table, (n, hkv, mk, d))
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
    return {"append": _exact_append, "attend": _exact_attend, "gather": _exact_gather}[case["op"]](s)


def _nearest_e4m3(x):
    """The nearest of e4m3's values, the even one of two: steps of 2^-3 of the power of two below, 2^-9 at least."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


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
        k, v = s["k"][cu[i]:cu[i + 1]].double(), s["v"][cu[i]:cu[i + 1]].double()
        for x, w in ((k, s["k_weight"]), (q[cu[i]:cu[i + 1]], s["q_weight"])):
            if w is not None:
                x *= w.double() / ((x ** 2).sum(2, keepdim=True) / c["d"] + EPS) ** 0.5
            y = torch.complex(x[..., first], x[..., second]) * z
            x[..., first], x[..., second] = y.real, y.imag
        if s["k_scale"] is not None:
            k = _nearest_e4m3(k / s["k_scale"].double()[None, :, None])
            v = _nearest_e4m3(v / s["v_scale"].double()[None, :, None])
        slot = s["block_table"][i][at // page].long()
        kc[slot, :, at % page] = k
        vc[slot, :, at % page] = v
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _tokens(s, i, a, b):
    """Keys and values of cached tokens [a, b) of request i: [tokens, heads, d]."""
    c, got = s["case"], []
    slots = s["block_table"][i][a // c["page"]:(b + c["page"] - 1) // c["page"]].long()
    a, b = a % c["page"], b - a // c["page"] * c["page"]
    for x, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        x = (x.view(torch.uint8)[slots].view(x.dtype) if scale is not None else x[slots]).double()
        x = x.transpose(1, 2).reshape(-1, c["hkv"], c["d"])[a:b]
        got.append(x if scale is None else x * scale.double()[None, :, None])
    return got


def _exact_gather(s):
    cu, first = s["cu_new"].tolist(), s["first"].tolist()
    k, v = zip(*(_tokens(s, i, f, f + cu[i + 1] - cu[i]) for i, f in enumerate(first)))
    return {"k": torch.cat(k), "v": torch.cat(v)}


def _exact_attend(s):
    c = s["case"]
    g = c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    cu, kv = s["cu_new"].tolist(), s["kv_len"].tolist()
    for i in range(c["n"]):
        a, b = cu[i], cu[i + 1]
        k, v = _tokens(s, i, 0, kv[i])
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
