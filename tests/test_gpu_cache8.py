"""GPU parity of kv_append_norm, kv_gather and paged_attention_fp8 against their
definitions in 64 bits."""
import numpy as np
import pytest

import cache8_reference as c8
from round_reference import BF16
from test_gpu_paged import APPEND, ATTEND, HIDDEN, _append_inputs, _cache, _cu, _i32, _lib  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.double().cpu().numpy()


def _f32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def _scales(rng, hkv):
    return _f32(rng.uniform(0.005, 0.03, hkv)), _f32(rng.uniform(0.005, 0.03, hkv))


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}[name]


def _as_bytes(c):
    """A cache to be compared bit for bit (NaN too)."""
    import torch
    return c.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[c.element_size()])


# ---------------------------------------------------------------------------
# kv_append_norm
# ---------------------------------------------------------------------------
def _check_append(new, kv, rot, inter, q, k, v, kc, vc, k_old, v_old, table, cs, q_out, kw, qw, eps, ks, vs, pos=None):
    import torch
    cu = _cu(new)
    T = int(cu[-1])
    place = np.concatenate([np.arange(kv[i] - n, kv[i]) for i, n in enumerate(new)])
    csr = _f64(cs)[place if pos is None else pos] if rot else np.zeros((T, 0))
    page, codes = kc.shape[2], kc.dtype == torch.float8_e4m3fn

    def formed(x, w):
        y, err = c8.norm(_f64(x), None if w is None else _f64(w), eps)
        return c8.rotate(y, err, csr, rot, inter)

    def near(got, want, err, dtype):
        half = 1.01 * BF16 * (np.abs(want) + err) if dtype == torch.bfloat16 else 0
        assert np.all(np.abs(got - want) <= err + half)

    slot = np.concatenate([[int(table[i, p // page]) for p in range(kv[i] - n, kv[i])] for i, n in enumerate(new)]).astype(int)
    row = place % page
    for got, old, (z, err), scale in ((kc, k_old, formed(k, kw), ks), (vc, v_old, (_f64(v), 0 * _f64(v)), vs)):
        at = torch.from_numpy(slot).cuda(), torch.from_numpy(row).cuda()
        mine = _f64(got.transpose(1, 2)[at] if not codes else _as_bytes(got).transpose(1, 2)[at].contiguous().view(got.dtype))
        if codes:
            s = np.ones(kc.shape[1]) if scale is None else _f64(scale)
            lo, hi = c8.code_range(z, err, s[None, :, None])
            assert np.all((lo <= mine) & (mine <= hi))
        else:
            near(mine, z, err, got.dtype)
        # and nothing else is written
        a, b = _as_bytes(got).transpose(1, 2).clone(), _as_bytes(old).transpose(1, 2).clone()
        a[at], b[at] = 0, 0
        assert torch.equal(a, b)
    if q_out is not None:
        near(_f64(q_out), *formed(q, qw), q_out.dtype)


NORM = APPEND + [
    ([9], [30], 3, 3, 1024, 1024, False, 4, "bf16", False),
    ([310, 20], [310, 20], 5, 1, 512, 128, True, 16, "bf16", True),
    ([1] * 33, [700 - 20 * i for i in range(33)], 10, 2, 128, 128, False, 16, "fp32", False),
    ([77], [200], 2, 2, 48, 16, False, 16, "bf16", False),
]


@pytest.mark.parametrize("new,kv,hq,hkv,d,rot,inter,page,dtype,tf", NORM)
@pytest.mark.parametrize("cache", ["e4m3", "own"])
@pytest.mark.parametrize("mode", ["q", "no q, positions", "no norm"])
def test_append_norm_parity(new, kv, hq, hkv, d, rot, inter, page, dtype, tf, cache, mode):
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(sum(kv) + d)
    dt = _dt(dtype)
    kc, vc, table = _cache(rng, new, kv, hkv, d, page, _dt("e4m3") if cache == "e4m3" else dt, tf)
    k_old, v_old = kc.clone(), vc.clone()
    q, k, v = _append_inputs(rng, new, hq, hkv, d, dt)
    cs = _f32(rng.normal(size=(max(kv) + 3, rot))) if rot else None
    T = int(np.sum(new))
    pos = rng.integers(0, max(kv) + 3, T).astype(np.int32) if "positions" in mode else None
    kw, qw = (_f32(rng.normal(1, 0.5, d)) for _ in range(2))
    if mode != "q":
        qw = None
    if mode == "no norm":
        kw = None
    ks, vs = _scales(rng, hkv) if cache == "e4m3" and mode != "no norm" else (None, None)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = svw.kv_append_norm(k, v, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), k_weight=kw, q_weight=qw, eps=1e-5,
                             k_scale=ks, v_scale=vs, cos_sin=cs, interleaved=inter,
                             positions=None if pos is None else _i32(pos), q=None if "no q" in mode else q, status=status)
    assert int(status) == 0 and (out is None) == ("no q" in mode)
    _check_append(new, kv, rot, inter, q, k, v, kc, vc, k_old, v_old, table, cs, out, kw, qw, 1e-5, ks, vs, pos)


@pytest.mark.parametrize("tokens,d", [(14, 64), (400, 64), (7, 128), (7, 40)])
@pytest.mark.parametrize("inter", [False, True])
def test_append_norm_queries_in_place(tokens, d, inter):
    import serving_vocab_wide_gb300 as svw
    rng = np.random.default_rng(2)
    new, kv = [tokens], [tokens + 30]
    kc, vc, table = _cache(rng, new, kv, 2, d, 16, _dt("e4m3"))
    k_old, v_old = kc.clone(), vc.clone()
    q, k, v = _append_inputs(rng, new, 4, 2, d, _dt("bf16"))
    q = q.contiguous()
    before = q.clone()
    cs, w = _f32(rng.normal(size=(tokens + 30, d))), _f32(rng.normal(1, 0.5, d))
    ks, vs = _scales(rng, 2)
    out = svw.kv_append_norm(k, v, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), k_weight=w, q_weight=w, eps=1e-6,
                             k_scale=ks, v_scale=vs, cos_sin=cs, interleaved=inter, q=q, q_out=q)
    assert out is q
    _check_append(new, kv, d, inter, before, k, v, kc, vc, k_old, v_old, table, cs, out, w, w, 1e-6, ks, vs)


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
def test_append_norm_misaligned_views(cache):
    """Strides and bases that no vector fits, of the tokens and of the caches."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(4)
    new, kv, hkv, d, page = [5, 9], [40, 9], 2, 64, 16
    _, _, table = _cache(rng, new, kv, hkv, d, page, _dt("bf16"))
    flat = torch.from_numpy(rng.normal(size=(14 * 900 + 7,))).to(torch.bfloat16).cuda()
    q = torch.as_strided(flat, (14, 4, d), (901, 65, 1), 1)
    k = torch.as_strided(flat, (14, hkv, d), (899, 67, 1), 300)
    v = torch.as_strided(flat, (14, hkv, d), (900, 66, 1), 501)
    n_pages = int(table.max()) + 1
    size = n_pages * 2300 + 50
    store = torch.zeros(2 * size, dtype=torch.uint8 if cache == "e4m3" else torch.bfloat16, device="cuda")
    strided = lambda i: torch.as_strided(store, (n_pages, hkv, page, d), (2300, 1131, 67, 1), i * size + 3)
    kc, vc = strided(0), strided(1)
    if cache == "e4m3":
        kc, vc = kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)
    k_old, v_old = kc.clone(), vc.clone()
    cs, w = _f32(rng.normal(size=(50, d))), _f32(rng.normal(1, 0.5, d))
    ks, vs = _scales(rng, hkv) if cache == "e4m3" else (None, None)
    out = svw.kv_append_norm(k, v, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), k_weight=w, q_weight=w, k_scale=ks,
                             v_scale=vs, cos_sin=cs, q=q)
    _check_append(new, kv, d, False, q, k, v, kc, vc, k_old, v_old, table, cs, out, w, w, 1e-6, ks, vs)


@pytest.mark.parametrize("tokens", [3, 400])
@pytest.mark.parametrize("d", [64, 40])
def test_append_norm_extremes(tokens, d):
    """Values beyond the codes' range, infinities, NaN, heads of zeros and ties."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(7)
    new, kv, hkv = [tokens], [tokens], 2
    kc, vc, table = _cache(rng, new, kv, hkv, d, 16, _dt("e4m3"))
    q, k, v = _append_inputs(rng, new, 2, hkv, d, _dt("bf16"))
    v = v.clone()
    v[0, 0, :8] = torch.tensor([1e30, -1e30, float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 464.0])
    v[0, 1, :8] = torch.tensor([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11, 448.0, -449.0, 432.0])
    k = k.clone()
    k[1] = 0
    k[2, 0, 1] = float("nan")
    svw.kv_append_norm(k, v, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), k_weight=_f32(np.ones(d)), eps=1e-6)
    got = vc[int(table[0, 0]), :, 0, :8].double().cpu().numpy()
    want = [[448, -448, 448, -448, np.nan, 0, 0, 448], [16, 20, 0, 2.0 ** -8, 0, 448, -448, 448]]
    assert np.array_equal(got, want, equal_nan=True)  # 17 and 19 lie between 16, 18 and 20
    row = kc[int(table[0, 0]), :, :3].double()
    assert bool((row[:, 1] == 0).all()) and bool(row[0, 2].isnan().all()) and not bool(row[1, 2].isnan().any())


@pytest.mark.parametrize("bad", [0.0, -1.0, float("nan"), float("inf"), 1e-40])
@pytest.mark.parametrize("tokens,d", [(2, 64), (330, 64), (2, 24)])
def test_append_norm_bad_scales(bad, tokens, d):
    """A scale that is no normal number > 0: its head's codes are NaN, the others as ever."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(9)
    new, kv, hkv = [tokens], [tokens], 3
    kc, vc, table = _cache(rng, new, kv, hkv, d, 16, _dt("e4m3"))
    q, k, v = _append_inputs(rng, new, 3, hkv, d, _dt("bf16"))
    ks, vs = _scales(rng, hkv)
    args = (_i32(table), _i32(_cu(new)), _i32(kv))
    good = kc.clone(), vc.clone()
    svw.kv_append_norm(k, v, *good, *args, k_scale=ks, v_scale=vs)
    k_bad, v_bad = ks.clone(), vs.clone()
    k_bad[1], v_bad[2] = bad, bad
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    svw.kv_append_norm(k, v, kc, vc, *args, k_scale=k_bad, v_scale=v_bad, status=status)
    assert int(status) == svw.SVW_DEV_BAD_INPUT
    for t in range(tokens):
        s, r = int(table[0, t // 16]), t % 16
        assert bool(kc[s, 1, r].double().isnan().all()) and bool(vc[s, 2, r].double().isnan().all())
    for c, g, h in ((kc, good[0], 1), (vc, good[1], 2)):
        a, b = _as_bytes(c).clone(), _as_bytes(g).clone()
        a[:, h], b[:, h] = 0, 0
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 24])
@pytest.mark.parametrize("many", [False, True])
def test_append_norm_bad_tokens_are_not_written(d, many):
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(6)
    new, kv, hkv, page = [3, 3, 3, 3] + [300] * many, [20, 2, 20, 20] + [300] * many, 2, 16
    kc, vc, table = _cache(rng, new, [20] * 4 + [300] * many, hkv, d, page, _dt("e4m3"))
    if not many:
        table = table[:, :2].copy()
    reach = table.shape[1] * page
    table[2, 1] = kc.shape[0]                                    # request 2: its second page is none of the cache's
    kv_dev = [20, 2, 20, reach + 2] + [300] * many               # 1: a negative place; 3: two tokens beyond the table
    table[3, -1] = table[3, 0] if many else table[3, 1]
    q, k, v = _append_inputs(rng, new, 2, hkv, d, _dt("bf16"))
    cs = _f32(rng.normal(size=(reach + 1, d)))
    k_old = _as_bytes(kc).clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = svw.kv_append_norm(k, v, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv_dev), cos_sin=cs, q=q, status=status)
    assert int(status) == svw.SVW_DEV_BAD_INPUT
    rows = {(int(p), int(r)) for p, _, r, _ in (_as_bytes(kc) != k_old).nonzero().tolist()}
    good = [(0, 17), (0, 18), (0, 19), (1, 0), (1, 1), (3, reach - 1)] + [(4, t) for t in range(300) if many]
    assert rows == {(int(table[i, p // page]), p % page) for i, p in good}
    nan = out.isnan().all(2).all(1).tolist()
    assert nan == [False] * 3 + [True, False, False] + [False] * 3 + [False, False, True] + [False] * 300 * many
    assert not bool(out.isnan().any(2).any(1)[~torch.tensor(nan, device="cuda")].any())


def test_append_norm_in_its_cache_is_append():
    """Without weights and codes it is kv_append, bit for bit."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(3)
    for new, kv, hq, hkv, d, rot, inter, page, dtype, tf in APPEND:
        kc, vc, table = _cache(rng, new, kv, hkv, d, page, _dt(dtype), tf)
        k2, v2 = kc.clone(), vc.clone()
        q, k, v = _append_inputs(rng, new, hq, hkv, d, _dt(dtype))
        cs = _f32(rng.normal(size=(max(kv), rot))) if rot else None
        rest = (_i32(table), _i32(_cu(new)), _i32(kv))
        a = svw.kv_append(k, v, kc, vc, *rest, cos_sin=cs, interleaved=inter, q=q)
        b = svw.kv_append_norm(k, v, k2, v2, *rest, cos_sin=cs, interleaved=inter, q=q)
        for x, y in ((a, b), (kc, k2), (vc, v2)):
            assert torch.equal(_as_bytes(x), _as_bytes(y))


# ---------------------------------------------------------------------------
# kv_gather
# ---------------------------------------------------------------------------
def _check_gather(n, first, table, c, scale, out):
    """Bit for bit the fp32 product, rounded once."""
    import torch
    cu, page, codes = _cu(n), c.shape[2], c.dtype == torch.float8_e4m3fn
    for i, m in enumerate(n):
        at = torch.arange(first[i], first[i] + m)
        slot = torch.from_numpy(table[i].astype(np.int64))[at // page].cuda()
        x = (_as_bytes(c) if codes else c)[slot, :, (at % page).cuda()].contiguous().view(c.dtype).float()
        want = x * scale[:, None] if scale is not None else x
        assert torch.equal(out[cu[i]:cu[i + 1]], want.to(out.dtype)), i


GATHER = [
    # tokens, first, heads, dim, page, tokens first
    ([1], [0], 1, 64, 16, False), ([777], [0], 8, 128, 16, False), ([5, 0, 300, 1], [3, 7, 0, 900], 2, 128, 64, True),
    ([33] * 50, list(range(50)), 3, 64, 32, False), ([9, 40], [1, 30], 2, 96, 24, False), ([200], [13], 5, 10, 7, True),
    ([64, 64], [64, 1], 1, 1024, 8, False), ([6], [5], 4, 48, 1, False), ([2000, 3], [1, 1999], 16, 256, 128, False),
]


@pytest.mark.parametrize("n,first,hkv,d,page,tf", GATHER)
@pytest.mark.parametrize("cache,out", [("e4m3", "bf16"), ("e4m3", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16"), ("fp32", "fp32")])
def test_gather_parity(n, first, hkv, d, page, tf, cache, out):
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(sum(n) + d)
    kc, vc, table = _cache(rng, n, [f + m for f, m in zip(first, n)], hkv, d, page, _dt(cache), tf)
    ks, vs = _scales(rng, hkv) if cache == "e4m3" else (None, None)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = svw.kv_gather(kc, vc, _i32(table), _i32(_cu(n)), first=_i32(first), k_scale=ks, v_scale=vs, dtype=_dt(out),
                         status=status)
    assert int(status) == 0
    _check_gather(n, first, table, kc, ks, k)
    _check_gather(n, first, table, vc, vs, v)


def test_gather_defaults_and_given_buffers():
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(2)
    n, hkv, d = [20, 7], 2, 64
    kc, vc, table = _cache(rng, n, n, hkv, d, 16, _dt("e4m3"))
    k, v = svw.kv_gather(kc, vc, _i32(table), _i32(_cu(n)))
    assert k.dtype == torch.bfloat16 and k.shape == (27, hkv, d)
    _check_gather(n, [0, 0], table, kc, None, k)
    # what lies behind the last token is left as it was, and an output may start anywhere
    store = torch.full((2, 28 * hkv * d + 1), 7.0, device="cuda")
    ko, vo = (s[1:1 + 27 * hkv * d].view(27, hkv, d) for s in store)
    a, b = svw.kv_gather(kc, vc, _i32(table), _i32(_cu(n)), k_out=ko, v_out=vo)
    assert a is ko and b is vo and torch.equal(ko, k.float()) and torch.equal(vo, v.float())
    assert bool((store[:, 0] == 7).all()) and bool((store[:, 1 + 27 * hkv * d:] == 7).all())
    none = svw.kv_gather(kc, vc, _i32(table), _i32([0, 0, 0]))
    assert none[0].shape == (0, hkv, d)


@pytest.mark.parametrize("d", [64, 24])
def test_gather_bad_tokens_and_scales(d):
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(5)
    n, first, hkv, page = [20, 20, 20, 20], [0, -1, 0, 30], 2, 16
    kc, vc, table = _cache(rng, n, [20, 20, 20, 50], hkv, d, page, _dt("e4m3"))
    table = table[:, :3].copy()        # request 3: its last two tokens lie beyond the table
    table[2, 1] = kc.shape[0]          # request 2: its second page is none of the cache's
    ks, vs = _scales(rng, hkv)
    cu = [0, 20, 40, 60, 80]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = svw.kv_gather(kc, vc, _i32(table), _i32(cu), first=_i32(first), k_scale=ks, v_scale=vs, status=status)
    assert int(status) == svw.SVW_DEV_BAD_INPUT
    bad = np.zeros(80, bool)
    bad[20:40] = bad[56:60] = bad[78:] = True
    for x in (k, v):
        assert np.array_equal(x.isnan().all(2).all(1).cpu().numpy(), bad)
        assert np.array_equal(x.isnan().any(2).any(1).cpu().numpy(), bad)
    # offsets that run backwards or beyond the outputs; a scale that is none
    status.zero_()
    k, _ = svw.kv_gather(kc, vc, _i32(table), _i32([0, 20, 10, 10, 10]), total_out=30, status=status)
    assert int(status) == svw.SVW_DEV_BAD_INPUT and bool(k[20:].isnan().all()) and not bool(k[:10].isnan().any())
    status.zero_()
    k, _ = svw.kv_gather(kc, vc, _i32(table), _i32([0, 10, 10, 10, 40]), total_out=30, status=status)
    assert int(status) == svw.SVW_DEV_BAD_INPUT and bool(k[10:].isnan().all()) and not bool(k[:10].isnan().any())
    status.zero_()
    ks[1] = 0
    k, v = svw.kv_gather(kc, vc, _i32(table[:1]), _i32([0, 20]), k_scale=ks, v_scale=vs, status=status)
    assert int(status) == svw.SVW_DEV_BAD_INPUT
    assert bool(k[:, 1].isnan().all()) and not bool(k[:, 0].isnan().any()) and not bool(v.isnan().any())


# ---------------------------------------------------------------------------
# paged_attention_fp8
# ---------------------------------------------------------------------------
def _dense(c, row, kv, scale):
    page = c.shape[2]
    slots = [int(s) for s in row[:-(-kv // page)]]
    x = _f64(_as_bytes(c)[slots].view(c.dtype)).transpose(0, 2, 1, 3).reshape(-1, c.shape[1], c.shape[3])[:kv]
    return x if scale is None else x * _f64(scale)[None, :, None]


def _compare_attend(new, kv, q, kc, vc, table, ks, vs, kw, out, lse, heads=None):
    hq, hkv, d = q.shape[1], kc.shape[1], kc.shape[3]
    cu = _cu(new)
    o, l, qd = _f64(out), _f64(lse), _f64(q)
    scale = float(np.float32(kw.get("scale", d ** -0.5)))
    worst = [0.0, 0.0]
    for i, n in enumerate(new):
        if n == 0:
            continue
        k, v = _dense(kc, table[i], max(0, kv[i]), ks), _dense(vc, table[i], max(0, kv[i]), vs)
        for h in range(hq) if heads is None else heads:
            hk = h // (hq // hkv)
            want, wl, bo, bl = c8.attend(qd[cu[i]:cu[i + 1], h], k[:, hk], v[:, hk], scale, kw.get("causal", True),
                                         kw.get("window", 0))
            go, gl = o[cu[i]:cu[i + 1], h], l[cu[i]:cu[i + 1], h]
            assert np.isfinite(go).all(), (i, h)
            none = np.isneginf(wl)
            assert np.array_equal(np.isneginf(gl), none), (i, h)
            assert np.all(go[none] == 0)
            worst[0] = max(worst[0], float(np.max(np.abs(go - want) / bo)))
            worst[1] = max(worst[1], float(np.max(np.abs(gl[~none] - wl[~none]) / bl[~none], initial=0)))
    assert worst[0] <= 1 and worst[1] <= 1, f"of the bounds: out {worst[0]}, lse {worst[1]}"


def _attend(new, kv, q, kc, vc, table, ks, vs, kw, status=None, **more):
    import serving_vocab_wide_gb300 as svw
    return svw.paged_attention_fp8(q, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), k_scale=ks, v_scale=vs,
                                   status=status, **kw, **more)


def _check_attend(new, kv, q, kc, vc, table, ks, vs, kw, heads=None):
    import torch
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _attend(new, kv, q, kc, vc, table, ks, vs, kw, status)
    assert int(status) == 0
    _compare_attend(new, kv, q, kc, vc, table, ks, vs, kw, out, lse, heads)
    return out, lse


def _codes(rng, new, kv, hkv, d, page, tf=False):
    """Caches of unit normal values (NaN where no request needs them) and their scales."""
    ks, vs = _scales(rng, hkv)
    kc, vc, table = _cache(rng, new, kv, hkv, d, page, _dt("fp32"), tf)
    code = lambda c, s: (c / s[None, :, None, None]).clamp(-448, 448).to(_dt("e4m3"))
    return code(kc, ks), code(vc, vs), table, ks, vs


def _queries(rng, new, hq, d, sd=1.5):
    import torch
    return torch.from_numpy(rng.normal(0, sd, size=(int(np.sum(new)), hq, d))).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("new,kv,hq,hkv,d,page,tf,kw", ATTEND)
def test_attend_fp8_parity(new, kv, hq, hkv, d, page, tf, kw):
    import torch
    rng = np.random.default_rng(sum(kv) + hq)
    kc, vc, table, ks, vs = _codes(rng, new, kv, hkv, d, page, tf)
    q = _queries(rng, new, hq, d)
    out, lse = _check_attend(new, kv, q, kc, vc, table, ks, vs, kw)
    again = _attend(new, kv, q, kc, vc, table, ks, vs, kw)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("n,kv,hq,hkv,d", [(1, 40000, 8, 2, 128), (17, 30011, 4, 1, 64), (64, 20000, 8, 2, 128)])
def test_attend_fp8_long_axis(n, kv, hq, hkv, d):
    import torch
    rng = np.random.default_rng(kv)
    kc, vc, table, ks, vs = _codes(rng, [n], [kv], hkv, d, 128)
    q = _queries(rng, [n], hq, d)
    out, lse = _check_attend([n], [kv], q, kc, vc, table, ks, vs, {}, heads=[0, hq - 1])
    again = _attend([n], [kv], q, kc, vc, table, ks, vs, {})
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("new,hq,d", [([20], 2, 64), ([20], 2, 128), ([200], 2, 64), ([200], 2, 128)])
def test_attend_fp8_large_scores(new, hq, d):
    """Scores whose running maximum keeps growing along the keys, by a lot and by a
    little, rows of equal scores, and queries of elements far apart."""
    import torch
    rng = np.random.default_rng(12)
    kv = [1500]
    kc, vc, table, ks, vs = _codes(rng, new, kv, 1, d, 16)
    ramp = (torch.linspace(0, 400, 1500, device="cuda")).to(_dt("e4m3"))
    for j in range(1500):
        kc[int(table[0, j // 16]), 0, j % 16, 0] = ramp[j]
    q = _queries(rng, new, hq, d, 1)
    q[:, 0, 0] = torch.linspace(-20, 20, new[0], device="cuda").to(torch.bfloat16)
    q[:, 1] = 0  # all scores equal: the mean of the values
    q[1::2, 1] = torch.exp2(torch.linspace(-40, 5, d, device="cuda")).to(torch.bfloat16)
    q[2::4] *= 1e-30
    _check_attend(new, kv, q, kc, vc, table, ks, vs, {"scale": 0.5})


def test_attend_fp8_without_scales_and_with_large_ones():
    import torch
    rng = np.random.default_rng(13)
    new, kv = [9, 150], [100, 700]
    for d in (64, 128):
        kc, vc, table, ks, vs = _codes(rng, new, kv, 2, d, 32)
        q = _queries(rng, new, 4, d)
        _check_attend(new, kv, q, kc, vc, table, None, None, {"scale": 0.001})
        _check_attend(new, kv, q, kc, vc, table, ks, None, {})
        ks2, vs2 = torch.full_like(ks, 2.0 ** 60), torch.full_like(vs, 2.0 ** -100)
        _check_attend(new, kv, q, kc, vc, table, ks2, vs2, {"scale": 2.0 ** -66})


def test_attend_fp8_strided_queries_and_given_buffers():
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(14)
    new, kv, hq, hkv, d = [6, 11], [300, 90], 6, 2, 128
    kc, vc, table, ks, vs = _codes(rng, new, kv, hkv, d, 32)
    qkv = torch.from_numpy(rng.normal(size=(17, (hq + 4) * d + 8))).to(torch.bfloat16).cuda()
    q = qkv[:, 8:8 + hq * d].view(17, hq, d)
    out = torch.empty(17, hq, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(17, hq, device="cuda")
    ws = torch.full((svw.paged_attention_workspace_size(17, hq, hkv, d),), 255, dtype=torch.uint8, device="cuda")
    got = _attend(new, kv, q, kc, vc, table, ks, vs, {}, out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse
    _compare_attend(new, kv, q, kc, vc, table, ks, vs, {}, out, lse)
    o2, none = _attend(new, kv, q, kc, vc, table, ks, vs, {}, want_lse=False)
    assert none is None and torch.equal(o2, out)
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)  # heads before tokens
    o3, _ = _attend(new, kv, qt, kc, vc, table, ks, vs, {})
    assert torch.equal(o3, out)


def test_attend_fp8_bad_requests():
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(16)
    new, kv, hq, hkv, d = [4, 4, 4, 4], [200, 200, 200, 200], 4, 2, 64
    kc, vc, table, ks, vs = _codes(rng, new, kv, hkv, d, 64)
    q = _queries(rng, new, hq, d)
    good = _attend(new, kv, q, kc, vc, table, ks, vs, {})
    for plant in (kc.shape[0], -1):
        t2, kv2 = table.copy(), list(kv)
        t2[1, 2] = plant                  # request 1: a page that is none of the cache's
        kv2[2] = table.shape[1] * 64 + 1  # request 2: more keys than its table holds
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = _attend(new, kv2, q, kc, vc, t2, ks, vs, {}, status)
        assert int(status) == svw.SVW_DEV_BAD_INPUT
        assert bool(out[4:12].isnan().all()) and bool(lse[4:12].isnan().all())
        for s in (slice(0, 4), slice(12, 16)):
            assert torch.equal(out[s], good[0][s]) and torch.equal(lse[s], good[1][s])


@pytest.mark.parametrize("new,kv", [([3, 1], [300, 20000]), ([9, 20], [300, 9000]), ([150, 40], [700, 300])])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_fp8_bad_scales_and_queries(new, kv, d):
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(17)
    hq, hkv = 6, 3
    kc, vc, table, ks, vs = _codes(rng, new, kv, hkv, d, 64)
    q = _queries(rng, new, hq, d)
    good = _attend(new, kv, q, kc, vc, table, ks, vs, {})
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-40):
        k2, v2 = ks.clone(), vs.clone()
        k2[0], v2[2] = bad, bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = _attend(new, kv, q, kc, vc, table, k2, v2, {}, status)
        assert int(status) == svw.SVW_DEV_BAD_INPUT
        assert bool(out[:, [0, 1, 4, 5]].isnan().all()) and bool(lse[:, :2].isnan().all())
        assert torch.equal(out[:, 2:4], good[0][:, 2:4]) and torch.equal(lse[:, 2:], good[1][:, 2:])
    q2 = q.clone()
    q2[0, 1, 3], q2[1, 2, d - 1], q2[2, 3, 0] = float("nan"), float("inf"), -float("inf")
    out, lse = _attend(new, kv, q2, kc, vc, table, ks, vs, {})
    odd = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    odd[0, 1] = odd[1, 2] = odd[2, 3] = True
    assert bool(out[odd].isnan().all()) and bool(lse[odd].isnan().all())
    assert torch.equal(out[~odd], good[0][~odd]) and torch.equal(lse[~odd], good[1][~odd])


@pytest.mark.parametrize("new,kv,hq,hkv,d,page,window", HIDDEN)
def test_attend_fp8_keys_behind_the_window_may_be_anything(new, kv, hq, hkv, d, page, window):
    import torch
    rng = np.random.default_rng(sum(kv) + d)
    kc, vc, table, ks, vs = _codes(rng, new, kv, hkv, d, page)
    q = _queries(rng, new, hq, d, 1)
    kw = {"window": window}
    clean = _check_attend(new, kv, q, kc, vc, table, ks, vs, kw)
    k2, v2, t2 = kc.clone(), vc.clone(), table.copy()
    hidden = 0
    for i, n in enumerate(new):
        unseen = max(0, kv[i] - n + 1 - window)  # before the first token's window
        for j in range(unseen):
            s, r = int(table[i, j // page]), j % page
            _as_bytes(k2)[s, :, r] = 0x7f
            _as_bytes(v2)[s, :, r] = 0xff if j % 2 else 0x7f
        t2[i, :unseen // page] = np.resize([-1, kc.shape[0] + 7, 1 << 30], unseen // page)
        hidden += unseen
    assert hidden > 0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _attend(new, kv, q, k2, v2, t2, ks, vs, kw, status)
    assert int(status) == 0
    assert torch.equal(lse, clean[1])
    _compare_attend(new, kv, q, kc, vc, table, ks, vs, kw, out, lse)


@pytest.mark.parametrize("new,kv,hq,hkv,d,page,window", HIDDEN)
@pytest.mark.parametrize("what", ["values", "keys"])
def test_attend_fp8_a_token_does_not_reach_those_before_it(new, kv, hq, hkv, d, page, window, what):
    """A later token's NaN reaches the tokens that see it, and no others."""
    import torch
    rng = np.random.default_rng(sum(kv) + d + 1)
    kc, vc, table, ks, vs = _codes(rng, new, kv, hkv, d, page)
    q = _queries(rng, new, hq, d, 1)
    k2, v2 = kc.clone(), vc.clone()
    cu = _cu(new)
    late = []
    for i, n in enumerate(new):
        j = kv[i] - (n + 1) // 2  # seen by the last half of the new tokens
        late.append(cu[i] + n - (n + 1) // 2)
        s, r = int(table[i, j // page]), j % page
        if what == "keys":
            _as_bytes(k2)[s, :, r, 1] = 0xff
        else:
            _as_bytes(v2)[s, :, r, 3] = 0x7f
    kw = {"window": window}
    out, lse = _attend(new, kv, q, k2, v2, table, ks, vs, kw)
    clean = _attend(new, kv, q, kc, vc, table, ks, vs, kw)
    got = out.clone()
    for i in range(len(new)):
        mine = got[late[i]:cu[i + 1]]
        if what == "keys":
            assert bool(mine.isnan().all()) and bool(lse[late[i]:cu[i + 1]].isnan().all())
            mine[:] = clean[0][late[i]:cu[i + 1]]
            lse[late[i]:cu[i + 1]] = clean[1][late[i]:cu[i + 1]]
        else:
            assert bool(mine[..., 3].isnan().all())
            mine[..., 3] = clean[0][late[i]:cu[i + 1], :, 3]
    _compare_attend(new, kv, q, kc, vc, table, ks, vs, kw, got, lse)


@pytest.mark.parametrize("new,kv,hq,hkv,d,page,first,window", [
    ([300], [2000], 8, 2, 128, 64, 1728, 0), ([300], [2000], 8, 2, 64, 16, 1840, 0),  # row tiles in pairs
    ([300], [2000], 8, 2, 128, 16, 1760, 100),
    ([40, 3], [2000, 100], 2, 2, 128, 16, 1984, 0), ([40, 3], [2000, 100], 2, 2, 64, 16, 1968, 20),
    ([17], [20000], 4, 1, 128, 16, 19984, 0),
    ([3], [20001], 4, 1, 128, 16, 20000, 0), ([3], [20000], 4, 1, 64, 64, 64, 19871)])  # joined by the last worker
def test_attend_fp8_a_bad_page_reaches_the_tokens_that_see_it(new, kv, hq, hkv, d, page, first, window):
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(first)
    kc, vc, table, ks, vs = _codes(rng, new, kv, hkv, d, page)
    q = _queries(rng, new, hq, d, 1)
    kw = {"window": window}
    good = _attend(new, kv, q, kc, vc, table, ks, vs, kw)
    at = kv[0] - new[0] + np.arange(new[0])
    sees = at >= first
    if window:
        sees &= at - window < first + page - 1
    assert sees.any() and not sees.all()
    sees = torch.from_numpy(np.concatenate([sees, np.zeros(sum(new[1:]), bool)])).cuda()
    for plant in (-1, kc.shape[0]):
        t2 = table.copy()
        t2[0, first // page] = plant
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = _attend(new, kv, q, kc, vc, t2, ks, vs, kw, status)
        assert int(status) == svw.SVW_DEV_BAD_INPUT
        assert bool(out[sees].isnan().all()) and bool(lse[sees].isnan().all())
        assert torch.equal(out[~sees], good[0][~sees]) and torch.equal(lse[~sees], good[1][~sees])


@pytest.mark.parametrize("new,kv,hq,hkv,d", [
    ([1], [9000], 8, 2, 128), ([1] * 5, [700, 1, 9000, 64, 3000], 8, 8, 64), ([17] * 6, [700, 1700, 9000, 64, 3000, 17], 8, 2, 128),
    ([17] * 6, [700, 1700, 9000, 64, 3000, 17], 8, 2, 64), ([300, 40], [3000, 900], 8, 2, 128), ([300, 40], [3000, 900], 8, 2, 64)])
def test_attend_fp8_streams_and_graphs(new, kv, hq, hkv, d):
    """Captured, replayed after cache, queries and scales have changed, and beside
    another stream's call: what a fresh call gives."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(26)
    kc, vc, table, ks, vs = _codes(rng, new, kv, hkv, d, 64)
    T = sum(new)
    q = _queries(rng, new, hq, d, 1)
    args = (q, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv))
    kw = dict(k_scale=ks, v_scale=vs)
    out, lse = torch.zeros_like(q), torch.zeros(T, hq, device="cuda")
    ws = torch.empty(svw.paged_attention_workspace_size(T, hq, hkv, d), dtype=torch.uint8, device="cuda")
    svw.paged_attention_fp8(*args, out=out, lse=lse, workspace=ws, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svw.paged_attention_fp8(*args, out=out, lse=lse, workspace=ws, **kw)
    side = torch.cuda.Stream()
    for n in range(10):
        _as_bytes(vc).bitwise_xor_(0x80)
        q.mul_(0.9)
        ks.mul_(1.01)
        torch.cuda.synchronize()
        g.replay()
        beside = svw.paged_attention_fp8(*args, stream=side, **kw)
        want = svw.paged_attention_fp8(*args, **kw)
        torch.cuda.synchronize()
        for o, l in ((out, lse), beside):
            assert torch.equal(o, want[0]) and torch.equal(l, want[1]), n
    _compare_attend(new, kv, q, kc, vc, table, ks, vs, {}, out, lse)


def test_two_graphs_share_a_workspace():
    """Captured calls that take turns with one workspace leave nothing in it that the other takes for its own."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(27)
    hq, hkv, d = 8, 2, 128
    ws, kept = None, []
    for new, kv in (([1], [9000]), ([3], [20000]), ([1, 1], [5000, 30])):
        kc, vc, table, ks, vs = _codes(rng, new, kv, hkv, d, 64)
        args = (_queries(rng, new, hq, d), kc, vc, _i32(table), _i32(_cu(new)), _i32(kv))
        kw = dict(k_scale=ks, v_scale=vs)
        if ws is None:
            ws = torch.empty(svw.paged_attention_workspace_size(8, hq, hkv, d), dtype=torch.uint8, device="cuda")
        kw |= dict(workspace=ws, out=torch.zeros_like(args[0]), lse=torch.zeros(sum(new), hq, device="cuda"))
        want = [t.clone() for t in svw.paged_attention_fp8(*args, **kw)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            svw.paged_attention_fp8(*args, **kw)
        kept.append((g, kw["out"], kw["lse"], want, args, ks, vs))
    for n in range(12):
        g, out, lse, want, *_ = kept[n * 5 % 3]
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_append_attend_gather_follow_on_one_stream():
    """What an append writes, the attention behind it reads, and a gather takes to
    another cache, call after call, as the context grows."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(20)
    hq, hkv, d, page = 4, 2, 128, 16
    steps = [[40, 3], [1, 1], [7, 17], [1, 0], [5, 2]]
    total = np.sum(steps, axis=0)
    kc, vc, table = _cache(rng, [0, 0], list(total), hkv, d, page, _dt("e4m3"))
    _as_bytes(kc).fill_(0x7f)
    _as_bytes(vc).fill_(0x7f)
    cs, kw, qw = _f32(rng.normal(size=(int(total.max()), d)) * 0.7), _f32(rng.normal(1, 0.3, d)), _f32(rng.normal(1, 0.3, d))
    ks, vs = _scales(rng, hkv)
    kv, kept, given = np.zeros(2, int), [], [[], []]
    for new in steps:
        kv = kv + new
        q, k, v = _append_inputs(rng, new, hq, hkv, d, _dt("bf16"))
        a = (_i32(table), _i32(_cu(new)), _i32(kv))
        qr = svw.kv_append_norm(k, v, kc, vc, *a, k_weight=kw, q_weight=qw, k_scale=ks, v_scale=vs, cos_sin=cs, q=q)
        out, lse = svw.paged_attention_fp8(qr, kc, vc, *a, k_scale=ks, v_scale=vs)
        kept.append((new, list(kv), qr, out, lse))
        for i, n in enumerate(new):
            given[i].append(v[_cu(new)[i]:_cu(new)[i] + n])
    for new, kv_then, qr, out, lse in kept:
        _compare_attend(new, kv_then, qr, kc, vc, table, ks, vs, {}, out, lse)
    # read back, the values are those that were given, to a code's rounding
    k, v = svw.kv_gather(kc, vc, _i32(table), _i32(_cu(kv)), k_scale=ks, v_scale=vs, dtype=torch.float32)
    want = torch.cat(given[0] + given[1]).float()
    step = 2.0 ** -9 * vs[:, None]
    clipped = want.clamp(-448 * vs[:, None], 448 * vs[:, None])
    assert bool(((v - clipped).abs() <= 1.001 * 2.0 ** -4 * clipped.abs() + 0.501 * step).all())
    # and written to a bf16 cache of other pages they give what the codes gave
    k16, v16, t16 = _cache(rng, [0, 0], list(kv), hkv, d, 64, _dt("bf16"))
    svw.kv_append(k.to(torch.bfloat16), v.to(torch.bfloat16), k16, v16, _i32(t16), _i32(_cu(kv)), _i32(kv))
    new, kv_then, qr, out, lse = kept[-1]
    o16, _ = svw.paged_attention(qr, k16, v16, _i32(t16), _i32(_cu(new)), _i32(kv))
    assert float((o16.float() - out.float()).norm() / out.float().norm()) < 2e-2  # keys within 2^-8 of the codes'


def test_beyond_32_bits_of_the_cache():
    """Pages whose bytes lie beyond 2^32 of the cache's start."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(8)
    hkv, d, page = 8, 128, 64
    n_pages = (1 << 32) // (hkv * d * page) + 40
    kc = torch.empty(n_pages, hkv, page, d, dtype=torch.float8_e4m3fn, device="cuda")
    vc = torch.empty_like(kc)
    new, kv = [200, 30], [200, 30]
    table = np.zeros((2, 4), np.int32)
    table[0] = n_pages - 1 - np.arange(4)
    table[1] = n_pages - 9 - np.arange(4)
    q, k, v = _append_inputs(rng, new, 8, hkv, d, _dt("bf16"))
    ks, vs = _scales(rng, hkv)
    rest = (_i32(table), _i32(_cu(new)))
    out = svw.kv_append_norm(k, v, kc, vc, *rest, _i32(kv), k_scale=ks, v_scale=vs, q=q)
    assert torch.equal(out, q)
    want = (k.float() / ks[:, None]).clamp(-448, 448)
    got, _ = svw.kv_gather(kc, vc, *rest, k_scale=ks, v_scale=vs, dtype=torch.float32)
    _check_gather(new, [0, 0], table, kc, ks, got)
    assert bool(((got / ks[:, None] - want).abs() <= 1.001 * 2.0 ** -4 * want.abs() + 2.0 ** -10 * 1.001).all())
    _check_attend(new, kv, out, kc, vc, table, ks, vs, {})


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 2, 64), (10, 2, 128), (5, 5, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_fp8_units_of_any_number_of_rows(hq, hkv, d, causal):
    """Requests of 1 to 33 tokens: row tiles on either side of the 64 rows up to
    which a CTA's second worker takes other lanes, many to a worker."""
    rng = np.random.default_rng(hq + d)
    new = [int(n) for n in rng.permutation(np.arange(1, 34)).repeat(3)]
    kv = [int(n + rng.integers(0, 700)) for n in new]
    kc, vc, table, ks, vs = _codes(rng, new, kv, hkv, d, 32)
    q = _queries(rng, new, hq, d)
    _check_attend(new, kv, q, kc, vc, table, ks, vs, {"causal": causal})


@pytest.mark.parametrize("n,kv,hq", [(1, 60000, 8), (20, 30000, 4), (150, 9000, 4)])
def test_attend_fp8_on_two_streams_without_a_wait(n, kv, hq):
    """Calls that make their own workspaces, in turn on the current stream and on
    another, the second before the first has ended: neither disturbs the other."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(n)
    kc, vc, table, ks, vs = _codes(rng, [n], [kv], 2, 128, 64)
    rest = (kc, vc, _i32(table), _i32([0, n]), _i32([kv]))
    qs = [_queries(rng, [n], hq, 128) for _ in range(2)]
    call = lambda q, **o: svw.paged_attention_fp8(q, *rest, k_scale=ks, v_scale=vs, **o)
    want = [call(q) for q in qs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        got = [call(qs[0]), call(qs[1], stream=side)]
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


@pytest.mark.parametrize("new,kv", [([1, 3], [40, 900]), ([300, 20, 1], [300, 500, 9])])
def test_append_norm_and_gather_captured_and_on_another_stream(new, kv):
    """Captured and replayed with other tokens, and on another stream: what fresh
    calls give."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(31)
    hq, hkv, d = 8, 2, 128
    kc, vc, table = _cache(rng, [0] * len(new), kv, hkv, d, 16, _dt("e4m3"), fill="nan")
    q, k, v = _append_inputs(rng, new, hq, hkv, d, _dt("bf16"))
    ks, vs = _scales(rng, hkv)
    w, cs = _f32(rng.normal(1, 0.3, d)), _f32(rng.normal(size=(max(kv), d)))
    where = (kc, vc, _i32(table))
    cu, lens, first = _i32(_cu(new)), _i32(kv), _i32([t - n for t, n in zip(kv, new)])
    qo = torch.empty_like(q)
    ko, vo = (torch.empty(sum(new), hkv, d, device="cuda") for _ in range(2))

    def both(stream=None, caches=where, out=(None, None, None)):
        kw = dict(k_scale=ks, v_scale=vs, stream=stream)
        r = svw.kv_append_norm(k, v, *caches, cu, lens, k_weight=w, q_weight=w, cos_sin=cs, q=q, q_out=out[0], **kw)
        return (r, *svw.kv_gather(*caches, cu, first=first, total_out=sum(new), dtype=torch.float32, k_out=out[1],
                                  v_out=out[2], **kw))

    both(out=(qo, ko, vo))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both(out=(qo, ko, vo))
    side = torch.cuda.Stream()
    for _ in range(4):
        for x in (q, k, v):
            x.mul_(-0.9)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        other = (torch.empty_like(kc), torch.empty_like(vc), where[2])
        fresh = both(caches=other)
        torch.cuda.synchronize()
        beside = both(stream=side, caches=other)
        torch.cuda.synchronize()
        for a, b, c in zip((qo, ko, vo), fresh, beside):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_gather_beyond_31_bits_of_the_outputs():
    """Outputs whose elements lie beyond 2^31, many tokens from one page."""
    import serving_vocab_wide_gb300 as svw
    import torch
    hkv, d, page = 16, 128, 16
    n = (1 << 31) // (hkv * d) + 50
    rng = np.random.default_rng(1)
    kc, vc, _ = _cache(rng, [0], [32], hkv, d, page, _dt("e4m3"))
    pages = -(-n // page)
    table = np.zeros((1, pages), np.int32)
    table[0, -2:] = [1, 0]
    kc[:2], vc[:2] = (torch.randn(2, hkv, page, d, device="cuda").to(_dt("e4m3")) for _ in range(2))
    k, v = svw.kv_gather(kc, vc, _i32(table), _i32([0, n]), total_out=n)
    for c, out in ((kc, k), (vc, v)):
        flat = c[:2].float().transpose(1, 2).to(torch.bfloat16)
        last = (pages - 2) * page
        assert torch.equal(out[last:last + page], flat[1]) and torch.equal(out[last + page:], flat[0][:n - last - page])
        assert torch.equal(out[:page], flat[0])


@pytest.mark.parametrize("new,kv", [([3, 1], [300, 70]), ([150, 40], [700, 300])])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_fp8_scores_that_vanish(new, kv, d):
    """Queries of zeros and scales so small that a score's factor would be zero:
    the hidden keys stay hidden, the weights of the others are equal."""
    import torch
    rng = np.random.default_rng(37)
    kc, vc, table, _, vs = _codes(rng, new, kv, 2, d, 32)
    q = _queries(rng, new, 4, d)
    q[::2] = 0
    q[1::2] *= 1e-37
    _check_attend(new, kv, q, kc, vc, table, torch.full((2,), 1e-30, device="cuda"), vs, {})


@pytest.mark.parametrize("new", [3, 150])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 12, -2.0 ** 12, 2.0 ** 15, -2.0 ** 15, 2.0 ** 100])
def test_attend_fp8_far_scores(new, d, size):
    """Scores of millions, thousands apart: the largest alone counts, however its
    maximum was reached; beyond what the call takes the rows are NaN."""
    import torch
    kv, page = 400, 16
    code = lambda *s: torch.zeros(*s, device="cuda").to(_dt("e4m3"))
    pages = -(-kv // page)
    kc, vc = code(pages, 1, page, d), code(pages, 1, page, d)
    up = torch.arange(pages * page, device="cuda").view(pages, 1, page)
    at = (448 - 32 * (up * 5 % 7)).float()  # up and down, in steps of e4m3's
    kc[..., 0] = at.to(_dt("e4m3"))
    best = at.max() if size > 0 else at.min()
    vc[..., :] = torch.where(at[..., None] == best, 2.0, 1.0).expand(vc.shape).to(_dt("e4m3"))
    q = torch.zeros(new, 2, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = size
    out, lse = _attend([new], [kv], q, kc, vc, np.arange(pages)[None].astype(np.int32), None, None,
                       {"scale": 1.0, "causal": False})
    top = float(best) * size
    if abs(top) > 2.9e6:
        assert bool(out.isnan().all()) and bool(lse.isnan().all())
    else:
        assert bool((out == 2).all()) and bool(((lse - top).abs() <= 2.0 ** -22 * abs(top) + 6).all())
