"""GPU parity of kv_append and paged_attention against their definitions in 64 bits."""
import numpy as np
import pytest

import round_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    import serving_vocab_wide_gb300 as svw
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    svw.build()
    svw.lib()


def _cache(rng, new, kv, hkv, d, page, dtype, tokens_first=False, spare=5, fill="nan"):
    """Pages handed out in a random order; what no request needs is NaN."""
    import torch
    need = [max(0, -(-k // page)) for k in kv]
    n_pages = sum(need) + spare
    order = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(new), max(need + [1]) + 2), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    shape = (n_pages, page, hkv, d) if tokens_first else (n_pages, hkv, page, d)
    caches = []
    for _ in range(2):
        c = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
        c = c.transpose(1, 2) if tokens_first else c
        caches.append(c)
    for i, k in enumerate(kv):
        for p in range(need[i]):
            rows = min(page, k - p * page)
            for c in caches:
                c[int(table[i, p]), :, :rows] = torch.from_numpy(rng.normal(size=(hkv, rows, d))).to(dtype).cuda()
    return caches[0], caches[1], table


def _dense(c, row, kv):
    """The first kv tokens of a request: float64 [kv, heads, dim]."""
    page = c.shape[2]
    slots = [int(s) for s in row[:-(-kv // page)]]
    return c[slots].double().cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, c.shape[1], c.shape[3])[:kv]


def _i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _cu(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


# ---------------------------------------------------------------------------
# kv_append
# ---------------------------------------------------------------------------
APPEND = [
    # new, kv_len, hq, hkv, d, rot, interleaved, page, dtype, tokens first
    ([1], [1], 4, 1, 64, 64, False, 16, "bf16", False),
    ([1, 0, 5, 33], [700, 9, 5, 100], 8, 2, 128, 128, False, 16, "bf16", False),
    ([1, 0, 5, 33], [700, 9, 5, 100], 8, 2, 128, 64, True, 64, "bf16", True),
    ([17, 2], [17, 300], 7, 7, 64, 64, True, 32, "fp32", False),
    ([3] * 40, [50 + 7 * i for i in range(40)], 5, 1, 128, 32, False, 128, "fp32", True),
    ([200, 1], [1000, 1], 6, 2, 80, 40, False, 24, "bf16", False),
    ([9], [30], 3, 3, 10, 6, False, 7, "bf16", True),
    ([9], [30], 3, 3, 10, 6, True, 1, "fp32", False),
    ([4, 4], [8, 4], 2, 1, 256, 256, False, 16, "bf16", False),
    ([6], [6], 2, 2, 64, 0, False, 16, "bf16", False),
    # many tokens, and heads whose slots are no power of two
    ([320, 7, 1], [320, 500, 77], 5, 2, 96, 32, False, 16, "bf16", False),
    ([330, 2], [600, 2], 9, 3, 80, 80, True, 32, "fp32", True),
    ([40, 300], [41, 300], 3, 1, 144, 48, False, 16, "bf16", False),
    ([310], [400], 12, 4, 1024, 512, False, 8, "fp32", False),
]


def _append_inputs(rng, new, hq, hkv, d, dt):
    import torch
    T = int(np.sum(new))
    qkv = torch.from_numpy(rng.normal(size=(T, (hq + 2 * hkv) * d))).to(dt).cuda()
    q = qkv[:, :hq * d].view(T, hq, d)
    k = qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
    v = qkv[:, (hq + hkv) * d:].view(T, hkv, d)
    return q, k, v


def _check_append(new, kv, rot, inter, q, k, v, kc, vc, k_old, v_old, table, cs, q_out, pos=None):
    import torch
    bf16 = kc.dtype == torch.bfloat16
    cu = _cu(new)
    T = int(cu[-1])
    place = np.concatenate([np.arange(kv[i] - n, kv[i]) for i, n in enumerate(new)]) if T else np.zeros(0, int)
    pos = place if pos is None else pos
    csr = cs.double().cpu().numpy()[pos] if rot else np.zeros((T, 0))
    f64 = lambda t: t.double().cpu().numpy()
    wk, sk = ref.rotate(f64(k), csr, rot, inter)
    want_k, want_v = f64(k_old), f64(v_old)
    bound = np.zeros_like(want_k)
    page = kc.shape[2]
    for i, n in enumerate(new):
        for t in range(n):
            p = kv[i] - n + t
            s, r = int(table[i, p // page]), p % page
            want_k[s, :, r], want_v[s, :, r] = wk[cu[i] + t], f64(v)[cu[i] + t]
            bound[s, :, r] = np.where(sk[cu[i] + t] > 0, ref.rotate_bound(wk[cu[i] + t], sk[cu[i] + t], bf16), 0)
    got_k, got_v = f64(kc), f64(vc)
    assert np.array_equal(np.isnan(got_k), np.isnan(want_k))
    assert np.all(np.nan_to_num(np.abs(got_k - want_k)) <= bound)
    assert np.array_equal(np.nan_to_num(got_v, nan=9e9), np.nan_to_num(want_v, nan=9e9))
    if q_out is not None:
        wq, sq = ref.rotate(f64(q), csr, rot, inter)
        assert np.all(np.abs(f64(q_out) - wq) <= np.where(sq > 0, ref.rotate_bound(wq, sq, bf16), 0))


@pytest.mark.parametrize("new,kv,hq,hkv,d,rot,inter,page,dtype,tf", APPEND)
@pytest.mark.parametrize("mode", ["q", "no q", "positions"])
def test_append_parity(new, kv, hq, hkv, d, rot, inter, page, dtype, tf, mode):
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(sum(kv) + d)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    kc, vc, table = _cache(rng, new, kv, hkv, d, page, dt, tf)
    k_old, v_old = kc.clone(), vc.clone()
    q, k, v = _append_inputs(rng, new, hq, hkv, d, dt)
    cs = torch.from_numpy(rng.normal(size=(max(kv) + 3, rot)).astype(np.float32)).cuda() if rot else None
    T = int(np.sum(new))
    pos = rng.integers(0, max(kv) + 3, T).astype(np.int32) if mode == "positions" else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = svw.kv_append(k, v, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), cos_sin=cs, interleaved=inter,
                        positions=None if pos is None else _i32(pos), q=None if mode == "no q" else q, status=status)
    assert int(status) == 0 and (out is None) == (mode == "no q")
    _check_append(new, kv, rot, inter, q, k, v, kc, vc, k_old, v_old, table, cs, out, pos)


@pytest.mark.parametrize("inter", [False, True])
def test_append_queries_in_place(inter):
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(2)
    new, kv = [5, 9], [40, 9]
    kc, vc, table = _cache(rng, new, kv, 2, 64, 16, torch.bfloat16)
    k_old, v_old = kc.clone(), vc.clone()
    q, k, v = _append_inputs(rng, new, 4, 2, 64, torch.bfloat16)
    q = q.contiguous()
    before = q.clone()
    cs = torch.from_numpy(rng.normal(size=(50, 64)).astype(np.float32)).cuda()
    out = svw.kv_append(k, v, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), cos_sin=cs, interleaved=inter, q=q, q_out=q)
    assert out is q
    _check_append(new, kv, 64, inter, before, k, v, kc, vc, k_old, v_old, table, cs, out)


def test_append_misaligned_views():
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(4)
    new, kv, hkv, d = [5, 9], [40, 9], 2, 64
    kc, vc, table = _cache(rng, new, kv, hkv, d, 16, torch.bfloat16)
    k_old, v_old = kc.clone(), vc.clone()
    flat = torch.from_numpy(rng.normal(size=(14 * 900 + 7,))).to(torch.bfloat16).cuda()
    q = torch.as_strided(flat, (14, 4, d), (901, 65, 1), 1)
    k = torch.as_strided(flat, (14, hkv, d), (899, 67, 1), 300)
    v = torch.as_strided(flat, (14, hkv, d), (900, 66, 1), 501)
    cs = torch.from_numpy(rng.normal(size=(50, d)).astype(np.float32)).cuda()
    out = svw.kv_append(k, v, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), cos_sin=cs, q=q)
    _check_append(new, kv, d, False, q, k, v, kc, vc, k_old, v_old, table, cs, out)


def test_append_bad_tokens_are_not_written():
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(6)
    new, kv, hkv, d, page = [3, 3, 3, 3], [20, 2, 20, 20], 2, 64, 16
    kc, vc, table = _cache(rng, [3] * 4, [20] * 4, hkv, d, page, torch.bfloat16)
    table = table[:, :2].copy()
    table[2, 1] = kc.shape[0]     # request 2: its second page is none of the cache's
    kv_dev = [20, 2, 20, 34]      # request 1: a negative place; request 3: two tokens beyond the table
    q, k, v = _append_inputs(rng, new, 2, hkv, d, torch.bfloat16)
    cs = torch.from_numpy(rng.normal(size=(33, d)).astype(np.float32)).cuda()
    k_old = kc.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = svw.kv_append(k, v, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv_dev), cos_sin=cs, q=q, status=status)
    assert int(status) == svw.SVW_DEV_BAD_INPUT
    changed = (kc != k_old) & ~(kc.isnan() & k_old.isnan())
    rows = {(int(p), int(r)) for p, _, r, _ in changed.nonzero().tolist()}
    good = [(0, 17), (0, 18), (0, 19), (1, 0), (1, 1), (3, 31)]
    assert rows == {(int(table[i, p // page]), p % page) for i, p in good}
    nan = out.isnan().all(2).all(1).tolist()
    assert nan == [False] * 3 + [True, False, False] + [False] * 3 + [False, False, True]


def test_append_beyond_32_bits_then_attend():
    """Pages whose elements lie beyond 2^31 of the cache's start."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(8)
    hkv, d, page = 8, 128, 64
    n_pages = (1 << 31) // (hkv * d * page) + 40
    kc = torch.empty(n_pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    new, kv = [200, 30], [200, 30]
    table = np.zeros((2, 4), np.int32)
    table[0] = n_pages - 1 - np.arange(4)
    table[1] = n_pages - 9 - np.arange(4)
    q, k, v = _append_inputs(rng, new, 8, hkv, d, torch.bfloat16)
    out = svw.kv_append(k, v, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), q=q)
    assert torch.equal(out, q)
    for i in range(2):
        a, b = _cu(new)[i], _cu(new)[i + 1]
        assert np.array_equal(_dense(kc, table[i], kv[i]), k[a:b].double().cpu().numpy())
        assert np.array_equal(_dense(vc, table[i], kv[i]), v[a:b].double().cpu().numpy())
    _check_attend(svw, new, kv, out, kc, vc, table, {})


# ---------------------------------------------------------------------------
# paged_attention
# ---------------------------------------------------------------------------
def _check_attend(svw, new, kv, q, kc, vc, table, kw, heads=None):
    import torch
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = svw.paged_attention(q, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), status=status, **kw)
    assert int(status) == 0
    _compare_attend(new, kv, q, kc, vc, table, kw, out, lse, heads)
    return out, lse


def _compare_attend(new, kv, q, kc, vc, table, kw, out, lse, heads=None):
    hq, hkv, d = q.shape[1], kc.shape[1], kc.shape[3]
    cu = _cu(new)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    qd = q.double().cpu().numpy()
    scale = float(np.float32(kw.get("scale", d ** -0.5)))
    worst = [0.0, 0.0]
    for i, n in enumerate(new):
        if n == 0:
            continue
        k, v = _dense(kc, table[i], max(0, kv[i])), _dense(vc, table[i], max(0, kv[i]))
        for h in range(hq) if heads is None else heads:
            hk = h // (hq // hkv)
            want, wl, bo, bl = ref.attend(qd[cu[i]:cu[i + 1], h], k[:, hk], v[:, hk], scale, kw.get("causal", True),
                                          kw.get("window", 0))
            go, gl = o[cu[i]:cu[i + 1], h], l[cu[i]:cu[i + 1], h]
            assert np.isfinite(go).all(), (i, h)
            none = np.isneginf(wl)
            assert np.array_equal(np.isneginf(gl), none), (i, h)
            assert np.all(go[none] == 0)
            worst[0] = max(worst[0], float(np.max(np.abs(go - want) / bo)))
            worst[1] = max(worst[1], float(np.max((np.abs(gl - wl) / bl)[~none], initial=0)))
    assert worst[0] <= 1 and worst[1] <= 1, f"of the bounds: out {worst[0]}, lse {worst[1]}"


ATTEND = [
    # new, kv_len, hq, hkv, d, page, tokens first, options
    ([1], [1], 1, 1, 64, 16, False, {}),
    ([1], [777], 32, 8, 128, 16, False, {}),
    ([1, 1, 1], [128, 129, 127], 8, 8, 128, 64, False, {}),
    ([3, 5, 17, 9], [3, 500, 1111, 64], 8, 2, 128, 32, False, {}),
    ([3, 5, 17, 9], [3, 500, 1111, 64], 8, 2, 64, 128, True, {}),
    ([17, 0, 33], [400, 50, 33], 7, 1, 128, 16, True, {"scale": 0.3}),
    ([16, 16], [16, 300], 5, 1, 64, 16, False, {"causal": False}),
    ([100, 130], [100, 1000], 4, 4, 128, 64, False, {}),
    ([300], [300], 8, 2, 128, 16, False, {}),
    ([129, 1], [900, 900], 6, 2, 64, 256, False, {"causal": False}),
    ([40, 1, 200], [600, 900, 200], 8, 2, 128, 32, False, {"window": 1}),
    ([40, 1, 200], [600, 900, 200], 8, 2, 128, 32, False, {"window": 130}),
    ([40, 1, 200], [600, 900, 200], 4, 4, 64, 16, True, {"window": 77}),
    ([2], [2], 64, 1, 128, 16, False, {}),
    ([9, 4], [700, 4], 128, 2, 64, 1024, False, {}),
    ([1] * 70, [1 + 13 * i for i in range(70)], 4, 2, 128, 16, False, {}),
    ([5, 3, 4], [2, 0, 4], 4, 2, 128, 16, False, {}),          # tokens at negative places see nothing
    ([5, 3], [0, 0], 4, 2, 64, 16, False, {"causal": False}),  # no keys at all
    ([260], [2000], 1, 1, 128, 64, False, {}),
    ([70, 70, 70], [70, 1500, 333], 3, 1, 64, 32, False, {"scale": 2.0}),
    # many tiles to a worker, and row tiles of which some or all rows have no token
    ([150, 45, 200], [4000, 3001, 5003], 8, 8, 64, 32, False, {}),
    ([150, 45, 200], [4000, 3001, 5003], 8, 8, 128, 16, False, {}),
    ([150, 45, 200], [4000, 3001, 5003], 8, 8, 64, 64, False, {"causal": False}),
    ([60, 3, 77], [5000, 4001, 3333], 20, 4, 64, 128, False, {"window": 2500}),
]


@pytest.mark.parametrize("new,kv,hq,hkv,d,page,tf,kw", ATTEND)
def test_attend_parity(new, kv, hq, hkv, d, page, tf, kw):
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(sum(kv) + hq)
    kc, vc, table = _cache(rng, new, kv, hkv, d, page, torch.bfloat16, tf)
    q = torch.from_numpy(rng.normal(0, 1.5, size=(int(np.sum(new)), hq, d))).to(torch.bfloat16).cuda()
    out, lse = _check_attend(svw, new, kv, q, kc, vc, table, kw)
    again = svw.paged_attention(q, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), **kw)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("n,kv,hq,hkv,d", [(1, 40000, 8, 2, 128), (17, 30011, 4, 1, 64), (64, 20000, 8, 2, 128)])
def test_attend_long_axis(n, kv, hq, hkv, d):
    """One request: the work is split over the keys and joined."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(kv)
    kc, vc, table = _cache(rng, [n], [kv], hkv, d, 128, torch.bfloat16)
    q = torch.from_numpy(rng.normal(0, 1.5, size=(n, hq, d))).to(torch.bfloat16).cuda()
    out, lse = _check_attend(svw, [n], [kv], q, kc, vc, table, {}, heads=[0, hq - 1])
    again = svw.paged_attention(q, kc, vc, _i32(table), _i32(_cu([n])), _i32([kv]))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_attend_large_scores():
    """Scores whose running maximum keeps growing along the keys, by a lot and
    by a little, and rows of equal scores."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(12)
    new, kv, hkv, d = [20], [1500], 1, 64
    kc, vc, table = _cache(rng, new, kv, hkv, d, 16, torch.bfloat16)
    ramp = torch.linspace(0, 30, 1500, device="cuda")
    for j in range(1500):
        kc[int(table[0, j // 16]), 0, j % 16, 0] = ramp[j]
    q = torch.from_numpy(rng.normal(0, 1, size=(20, 2, d))).to(torch.bfloat16).cuda()
    q[:, 0, 0] = torch.linspace(-20, 20, 20, device="cuda").to(torch.bfloat16)
    q[:, 1] = 0  # all scores equal: the mean of the values
    _check_attend(svw, new, kv, q, kc, vc, table, {"scale": 0.5})


def test_attend_strided_queries_and_given_buffers():
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(14)
    new, kv, hq, hkv, d = [6, 11], [300, 90], 6, 2, 128
    kc, vc, table = _cache(rng, new, kv, hkv, d, 32, torch.bfloat16)
    qkv = torch.from_numpy(rng.normal(size=(17, (hq + 4) * d + 8))).to(torch.bfloat16).cuda()
    q = qkv[:, 8:8 + hq * d].view(17, hq, d)
    out = torch.empty(17, hq, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(17, hq, device="cuda")
    ws = torch.full((svw.paged_attention_workspace_size(17, hq, hkv, d),), 255, dtype=torch.uint8, device="cuda")
    got = svw.paged_attention(q, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse
    _compare_attend(new, kv, q, kc, vc, table, {}, out, lse)
    o2, none = svw.paged_attention(q, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), want_lse=False)
    assert none is None and torch.equal(o2, out)
    # heads before tokens
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    o3, _ = svw.paged_attention(qt, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv))
    assert torch.equal(o3, out)


def test_attend_bad_requests():
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(16)
    new, kv, hq, hkv, d = [4, 4, 4, 4], [200, 200, 200, 200], 4, 2, 64
    kc, vc, table = _cache(rng, new, kv, hkv, d, 64, torch.bfloat16)
    q = torch.from_numpy(rng.normal(size=(16, hq, d))).to(torch.bfloat16).cuda()
    good = svw.paged_attention(q, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv))
    for plant in (kc.shape[0], -1):
        t2, kv2 = table.copy(), list(kv)
        t2[1, 2] = plant                  # request 1: a page that is none of the cache's
        kv2[2] = table.shape[1] * 64 + 1  # request 2: more keys than its table holds
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = svw.paged_attention(q, kc, vc, _i32(t2), _i32(_cu(new)), _i32(kv2), status=status)
        assert int(status) == svw.SVW_DEV_BAD_INPUT
        assert bool(out[4:12].isnan().all()) and bool(lse[4:12].isnan().all())
        for s in (slice(0, 4), slice(12, 16)):
            assert torch.equal(out[s], good[0][s]) and torch.equal(lse[s], good[1][s])


HIDDEN = [
    # new, kv_len, hq, hkv, d, page, window: decoding, blocks, prompts, one long request
    ([1, 1, 1], [700, 130, 64], 8, 2, 128, 16, 70),
    ([17, 5], [900, 200], 4, 4, 64, 16, 33),
    ([17, 5], [900, 200], 8, 1, 128, 64, 100),
    ([150, 40], [700, 300], 4, 2, 64, 32, 90),
    ([150, 40], [700, 300], 4, 2, 128, 16, 200),
    ([9], [20000], 4, 1, 128, 16, 7000),
]


@pytest.mark.parametrize("new,kv,hq,hkv,d,page,window", HIDDEN)
def test_attend_keys_behind_the_window_may_be_anything(new, kv, hq, hkv, d, page, window):
    """What no token sees changes nothing: NaN, infinities, and the block
    table's entries of pages that lie behind every token's window."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(sum(kv) + d)
    kc, vc, table = _cache(rng, new, kv, hkv, d, page, torch.bfloat16)
    q = torch.from_numpy(rng.normal(size=(int(np.sum(new)), hq, d))).to(torch.bfloat16).cuda()
    kw = {"window": window}
    clean = _check_attend(svw, new, kv, q, kc, vc, table, kw)
    k2, v2, t2 = kc.clone(), vc.clone(), table.copy()
    hidden = 0
    for i, n in enumerate(new):
        unseen = max(0, kv[i] - n + 1 - window)  # before the first token's window
        for j in range(unseen):
            s, r = int(table[i, j // page]), j % page
            k2[s, :, r] = float("nan")
            v2[s, :, r] = float("nan") if j % 2 else float("inf")
        t2[i, :unseen // page] = np.resize([-1, kc.shape[0] + 7, 1 << 30], unseen // page)
        hidden += unseen
    assert hidden > 0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = svw.paged_attention(q, k2, v2, _i32(t2), _i32(_cu(new)), _i32(kv), status=status, **kw)
    assert int(status) == 0
    assert torch.equal(lse, clean[1])
    _compare_attend(new, kv, q, kc, vc, table, kw, out, lse)


@pytest.mark.parametrize("new,kv,hq,hkv,d,page,window", HIDDEN)
@pytest.mark.parametrize("what", ["values", "keys"])
def test_attend_a_token_does_not_reach_those_before_it(new, kv, hq, hkv, d, page, window, what):
    """A later token's NaN or infinity reaches the tokens that see it, and no
    others."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(sum(kv) + d + 1)
    kc, vc, table = _cache(rng, new, kv, hkv, d, page, torch.bfloat16)
    q = torch.from_numpy(rng.normal(size=(int(np.sum(new)), hq, d))).to(torch.bfloat16).cuda()
    k2, v2 = kc.clone(), vc.clone()
    cu = _cu(new)
    late = []
    for i, n in enumerate(new):
        j = kv[i] - (n + 1) // 2  # seen by the last half of the new tokens
        late.append(cu[i] + n - (n + 1) // 2)
        s, r = int(table[i, j // page]), j % page
        if what == "keys":
            k2[s, :, r, 1] = float("nan")
        else:
            v2[s, :, r, 3] = float("nan")
            v2[s, :, r, 5] = float("inf")
    out, lse = svw.paged_attention(q, k2, v2, _i32(table), _i32(cu), _i32(kv), window=window)
    clean = svw.paged_attention(q, kc, vc, _i32(table), _i32(cu), _i32(kv), window=window)
    got = out.clone()
    for i, n in enumerate(new):
        mine = got[late[i]:cu[i + 1]]
        seen = torch.arange(mine.shape[0]) < window  # the token itself leaves the window again
        assert bool(seen.all())
        if what == "keys":
            assert bool(mine.isnan().all()) and bool(lse[late[i]:cu[i + 1]].isnan().all())
            mine[:] = clean[0][late[i]:cu[i + 1]]
            lse[late[i]:cu[i + 1]] = clean[1][late[i]:cu[i + 1]]
        else:
            assert bool(mine[..., 3].isnan().all()) and bool(torch.isposinf(mine[..., 5]).all())
            for e in (3, 5):
                mine[..., e] = clean[0][late[i]:cu[i + 1], :, e]
    _compare_attend(new, kv, q, kc, vc, table, {"window": window}, got, lse)


def test_attend_streams_and_graph():
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(18)
    new, kv, hq, hkv, d = [5, 1], [2000, 900], 8, 2, 128
    kc, vc, table = _cache(rng, new, kv, hkv, d, 64, torch.bfloat16)
    q = torch.from_numpy(rng.normal(size=(6, hq, d))).to(torch.bfloat16).cuda()
    args = (q, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv))
    want = svw.paged_attention(*args)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = [svw.paged_attention(*args, stream=s) for s in (a, b, a, b)]
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    ws = torch.empty(svw.paged_attention_workspace_size(6, hq, hkv, d), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svw.paged_attention(*args, out=out, lse=lse, workspace=ws)
    for _ in range(3):  # one captured call, replayed: the same workspace as it was left
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("new,kv,hq,hkv", [([1], [9000], 8, 2), ([1] * 5, [700, 1, 9000, 64, 3000], 8, 8), ([2], [30000], 4, 1)])
def test_attend_replays_with_other_keys(new, kv, hq, hkv):
    """A captured call of few rows, replayed after its cache has changed, gives
    what a fresh call gives: nothing of an earlier replay is joined in."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(24)
    kc, vc, table = _cache(rng, new, kv, hkv, 128, 64, torch.bfloat16)
    T = sum(new)
    q = torch.from_numpy(rng.normal(size=(T, hq, 128))).to(torch.bfloat16).cuda()
    args = (q, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv))
    out, lse = torch.zeros_like(q), torch.zeros(T, hq, device="cuda")
    ws = torch.empty(svw.paged_attention_workspace_size(T, hq, hkv, 128), dtype=torch.uint8, device="cuda")
    svw.paged_attention(*args, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svw.paged_attention(*args, out=out, lse=lse, workspace=ws)
    for n in range(20):
        vc.mul_(-1)
        q.mul_(0.9)
        g.replay()
        want = svw.paged_attention(*args)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), n


def test_append_then_attend_follow_on_one_stream():
    """What an append writes, the attention behind it reads, call after call,
    as the context grows."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(20)
    hq, hkv, d, page = 4, 2, 128, 16
    steps = [[40, 3], [1, 1], [7, 17], [1, 0], [5, 2]]
    total = np.sum(steps, axis=0)
    kc, vc, table = _cache(rng, [0, 0], list(total), hkv, d, page, torch.bfloat16)
    kc.fill_(float("nan"))
    vc.fill_(float("nan"))
    cs = torch.from_numpy(rng.normal(size=(int(total.max()), d)).astype(np.float32) * 0.7).cuda()
    kv, kept = np.zeros(2, int), []
    for new in steps:
        kv = kv + new
        q, k, v = _append_inputs(rng, new, hq, hkv, d, torch.bfloat16)
        a = (_i32(table), _i32(_cu(new)), _i32(kv))
        qr = svw.kv_append(k, v, kc, vc, *a, cos_sin=cs, q=q)
        out, lse = svw.paged_attention(qr, kc, vc, *a)
        kept.append((new, list(kv), qr, out, lse))
    for new, kv_then, qr, out, lse in kept:
        _compare_attend(new, kv_then, qr, kc, vc, table, {}, out, lse)


def test_paged_refusals():
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(22)
    new, kv, hq, hkv, d = [4, 4], [100, 30], 4, 2, 64
    kc, vc, table = _cache(rng, new, kv, hkv, d, 16, torch.bfloat16)
    q, k, v = _append_inputs(rng, new, hq, hkv, d, torch.bfloat16)
    tb, cu, kl = _i32(table), _i32(_cu(new)), _i32(kv)
    cs = torch.zeros(200, d, device="cuda")
    E = svw.SvwError
    app = lambda **o: svw.kv_append(*[o.pop(n, x) for n, x in (("k", k), ("v", v), ("k_cache", kc), ("v_cache", vc),
                                    ("block_table", tb), ("cu_new", cu), ("kv_len", kl))], **o)
    for o in ({"k": k.float()}, {"k": k[:, :1]}, {"v": v[:-1]}, {"cu_new": cu.long()}, {"kv_len": kl[:1]},
              {"block_table": tb[:1]}, {"block_table": tb.long()}, {"cos_sin": cs.double()}, {"cos_sin": cs[:, :63].contiguous()},
              {"cos_sin": torch.zeros(9, 2 * d, device="cuda")}, {"q": q[:-1]}, {"q": q.float()}, {"q_out": q},
              {"q": q, "q_out": q}, {"v_cache": vc[:, :1]}, {"positions": cu}, {"k_cache": kc.cpu()},
              {"k_cache": kc.half(), "v_cache": vc.half(), "k": k.half(), "v": v.half()}):
        with pytest.raises(E):
            app(**o)
    att = lambda **o: svw.paged_attention(*[o.pop(n, x) for n, x in (("q", q), ("k_cache", kc), ("v_cache", vc),
                                          ("block_table", tb), ("cu_new", cu), ("kv_len", kl))], **o)
    f = torch.zeros(4, 2, 16, 64, device="cuda")
    p24 = torch.zeros(4, 2, 24, 64, dtype=torch.bfloat16, device="cuda")
    d96 = torch.zeros(4, 2, 16, 96, dtype=torch.bfloat16, device="cuda")
    one = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    for o in ({"q": q[:, :3]}, {"q": q.float()}, {"q": q.float(), "k_cache": f, "v_cache": f}, {"scale": 0.0},
              {"scale": -1.0}, {"scale": float("inf")}, {"scale": float("nan")}, {"window": -1},
              {"window": 5, "causal": False}, {"k_cache": p24, "v_cache": p24},
              {"q": torch.zeros(8, 4, 96, dtype=torch.bfloat16, device="cuda"), "k_cache": d96, "v_cache": d96},
              {"q": torch.zeros(8, 65, 64, dtype=torch.bfloat16, device="cuda"), "k_cache": one, "v_cache": one},
              {"q": q[:1].expand(8, hq, d)}, {"out": torch.zeros(8, hq, d, device="cuda")},
              {"lse": torch.zeros(7, hq, device="cuda")},
              {"workspace": torch.zeros(0, dtype=torch.uint8, device="cuda")}, {"kv_len": kl.long()}):
        with pytest.raises(E):
            att(**o)
    # a base that is not 16-byte aligned
    flat = torch.zeros(8 * hq * d + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(E):
        att(q=flat[1:1 + 8 * hq * d].view(8, hq, d))
    # nothing to do is fine
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = att(q=q[:0], cu_new=none)
    assert out.shape == (0, hq, d) and lse.shape == (0, hq)
    assert app(k=k[:0], v=v[:0], cu_new=none) is None


@pytest.mark.parametrize("n,kv,hq", [(1, 60000, 8), (20, 30000, 4), (150, 9000, 4)])
def test_attend_on_two_streams_without_a_wait(n, kv, hq):
    """Calls that make their own workspaces, in turn on the current stream and on
    another, the second before the first has ended: neither disturbs the other."""
    import serving_vocab_wide_gb300 as svw
    import torch
    g = torch.Generator(device="cuda").manual_seed(kv)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    pages = -(-kv // 64)
    rest = (r(pages, 2, 64, 128), r(pages, 2, 64, 128), _i32(np.arange(pages)[None]), _i32([0, n]), _i32([kv]))
    qs = [r(n, hq, 128) for _ in range(2)]
    want = [svw.paged_attention(q, *rest) for q in qs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        got = [svw.paged_attention(qs[0], *rest), svw.paged_attention(qs[1], *rest, stream=side)]
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


@pytest.mark.parametrize("hkv,d,rot,dtype", [(2, 64, 32, "bf16"), (1, 128, 64, "fp32"), (3, 10, 6, "fp32"), (3, 10, 4, "bf16")])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("tokens", [3, 400])
def test_append_a_query_without_a_position_is_nan(hkv, d, rot, dtype, inter, tokens):
    """All of it, the elements that are not rotated too; its key and value are not
    written, the other tokens are as ever."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(d + rot)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    new, kv = [tokens], [tokens + 20]
    kc, vc, table = _cache(rng, new, kv, hkv, d, 16, dt)
    q, k, v = _append_inputs(rng, new, 2 * hkv, hkv, d, dt)
    cs = torch.from_numpy(rng.normal(size=(40, rot)).astype(np.float32)).cuda()
    pos = rng.integers(0, 40, tokens).astype(np.int32)
    pos[[0, tokens // 2]] = [40, -1]
    k_old, v_old = kc.clone(), vc.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = svw.kv_append(k, v, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), cos_sin=cs, interleaved=inter,
                        positions=_i32(pos), q=q, status=status)
    assert int(status) == svw.SVW_DEV_BAD_INPUT
    bad = torch.from_numpy((pos < 0) | (pos >= 40)).cuda()
    assert bool(out[bad].isnan().all()) and not bool(out[~bad].isnan().any())
    for t in torch.nonzero(bad).flatten().tolist():
        s, r = int(table[0, (20 + t) // 16]), (20 + t) % 16
        assert torch.equal(kc[s, :, r], k_old[s, :, r]) and torch.equal(vc[s, :, r], v_old[s, :, r])
    good = svw.kv_append(k, v, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), cos_sin=cs, interleaved=inter,
                         positions=_i32(np.clip(pos, 0, 39)), q=q)
    assert torch.equal(out[~bad], good[~bad])


@pytest.mark.parametrize("new,kv,hq,hkv,d,page,first,window", [
    ([300], [2000], 8, 2, 128, 64, 1728, 0), ([300], [2000], 8, 2, 64, 16, 1840, 0),  # row tiles in pairs
    ([300], [2000], 8, 2, 128, 16, 1760, 100),
    ([40, 3], [2000, 100], 2, 2, 128, 16, 1984, 0), ([40, 3], [2000, 100], 2, 2, 64, 16, 1968, 20),
    ([17], [20000], 4, 1, 128, 16, 19984, 0),
    ([3], [20001], 4, 1, 128, 16, 20000, 0), ([3], [20000], 4, 1, 64, 64, 64, 19871)])  # joined by the last worker
def test_attend_a_bad_page_reaches_the_tokens_that_see_it(new, kv, hq, hkv, d, page, first, window):
    """The page of places first .. first + page - 1 of request 0 is none of the
    cache's: tokens that see one of them are NaN, the others as with a good page."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(first)
    kc, vc, table = _cache(rng, new, kv, hkv, d, page, torch.bfloat16)
    q = torch.from_numpy(rng.normal(size=(int(np.sum(new)), hq, d))).to(torch.bfloat16).cuda()
    rest = (_i32(_cu(new)), _i32(kv))
    good = svw.paged_attention(q, kc, vc, _i32(table), *rest, window=window)
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
        out, lse = svw.paged_attention(q, kc, vc, _i32(t2), *rest, window=window, status=status)
        assert int(status) == svw.SVW_DEV_BAD_INPUT
        assert bool(out[sees].isnan().all()) and bool(lse[sees].isnan().all())
        assert torch.equal(out[~sees], good[0][~sees]) and torch.equal(lse[~sees], good[1][~sees])


@pytest.mark.parametrize("T,hq", [(1, 4), (9, 1), (1, 1)])
def test_append_queries_in_place_where_a_dimension_is_one(T, hq):
    """A split of one token's projection, or of one head, is contiguous whatever
    its strides say of that dimension: rotated in place as any other."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(T + hq)
    d, kv = 64, [30]
    kc, vc, table = _cache(rng, [T], kv, 1, d, 16, torch.bfloat16)
    qkv = torch.from_numpy(rng.normal(size=(T, (hq + 2) * d))).to(torch.bfloat16).cuda()
    k, v = qkv[:, hq * d:(hq + 1) * d].view(T, 1, d), qkv[:, (hq + 1) * d:].view(T, 1, d)
    q = qkv[:, :hq * d].view(T, hq, d)
    if T > 1:
        q = torch.as_strided(q.contiguous(), (T, hq, d), (hq * d, 7, 1))
    assert q.is_contiguous()
    cs = torch.from_numpy(rng.normal(size=(40, d)).astype(np.float32)).cuda()
    where = (_i32(table), _i32(_cu([T])), _i32(kv))
    want = svw.kv_append(k, v, kc, vc, *where, cos_sin=cs, q=q.clone())
    out = svw.kv_append(k, v, kc, vc, *where, cos_sin=cs, q=q, q_out=q)
    assert out is q and torch.equal(out, want)


def test_append_a_range_beyond_the_tokens_is_not_written():
    """A request whose new tokens would end behind the last one given is bad, as it
    is for paged_attention: none of it is written, the others are."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(5)
    kc, vc, table = _cache(rng, [3, 5], [20, 20], 2, 64, 16, torch.bfloat16)
    q, k, v = _append_inputs(rng, [3, 3], 4, 2, 64, torch.bfloat16)
    k_old = kc.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = svw.kv_append(k, v, kc, vc, _i32(table), _i32([0, 3, 8]), _i32([20, 20]), q=q, status=status)
    assert int(status) == svw.SVW_DEV_BAD_INPUT and torch.equal(out, q)  # no rotation
    changed = (kc != k_old) & ~(kc.isnan() & k_old.isnan())
    rows = {(int(p), int(r)) for p, _, r, _ in changed.nonzero().tolist()}
    assert rows == {(int(table[0, p // 16]), p % 16) for p in (17, 18, 19)}
    assert np.array_equal(_dense(kc, table[0], 20)[17:], k[:3].double().cpu().numpy())


@pytest.mark.parametrize("new,kv,hq,hkv,d", [
    ([17] * 6, [700, 1700, 9000, 64, 3000, 17], 8, 2, 128), ([17] * 6, [700, 1700, 9000, 64, 3000, 17], 8, 2, 64),
    ([300, 40], [3000, 900], 8, 2, 128), ([300, 40], [3000, 900], 8, 2, 64)])
def test_attend_joined_apart_replays_with_other_keys(new, kv, hq, hkv, d):
    """The same with the join as a kernel of its own: captured, replayed after the
    cache has changed, and beside another stream's call."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(26)
    kc, vc, table = _cache(rng, new, kv, hkv, d, 64, torch.bfloat16)
    T = sum(new)
    q = torch.from_numpy(rng.normal(size=(T, hq, d))).to(torch.bfloat16).cuda()
    args = (q, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv))
    out, lse = torch.zeros_like(q), torch.zeros(T, hq, device="cuda")
    ws = torch.empty(svw.paged_attention_workspace_size(T, hq, hkv, d), dtype=torch.uint8, device="cuda")
    svw.paged_attention(*args, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svw.paged_attention(*args, out=out, lse=lse, workspace=ws)
    side = torch.cuda.Stream()
    for n in range(10):
        vc.mul_(-1)
        q.mul_(0.9)
        torch.cuda.synchronize()
        g.replay()
        beside = svw.paged_attention(*args, stream=side)
        want = svw.paged_attention(*args)
        torch.cuda.synchronize()
        for o, l in ((out, lse), beside):
            assert torch.equal(o, want[0]) and torch.equal(l, want[1]), n
    _compare_attend(new, kv, q, kc, vc, table, {}, out, lse)
