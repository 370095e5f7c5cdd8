"""kv_append_norm, kv_gather and paged_attention_fp8 at the ends of what they accept."""
import math

import numpy as np
import pytest

from test_gpu_cache8 import _as_bytes, _attend, _codes, _compare_attend, _f32, _queries
from test_gpu_paged import _append_inputs, _cache, _cu, _i32, _lib  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

FLT_MIN, FLT_MAX = 2.0 ** -126, float(np.finfo(np.float32).max)


# ---------------------------------------------------------------------------
# paged_attention_fp8
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("new,kv,causal", [
    ([2, 3], [0, 40], True), ([4, 1], [2, 300], True), ([100], [99], True), ([300], [299], True), ([2, 3], [0, 40], False),
    ([300, 2], [0, 40], False)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_bad_scale_reaches_rows_that_see_no_key(new, kv, causal, d):
    """Rows without keys are 0 and -inf, and NaN like all others under a scale that is none."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(d + sum(kv))
    hq, hkv = 6, 3
    kc, vc, table, ks, vs = _codes(rng, new, kv, hkv, d, 16)
    q = _queries(rng, new, hq, d)
    kw = {"causal": causal}
    good = _attend(new, kv, q, kc, vc, table, ks, vs, kw)
    place = np.concatenate([np.arange(k - n, k) if causal else np.full(n, k - 1) for n, k in zip(new, kv)])
    none = torch.from_numpy(place < 0).cuda()
    assert bool(none.any()) and bool((good[0][none] == 0).all()) and bool((good[1][none] == -math.inf).all())
    for bad in (0.0, float("nan"), float("inf"), 1e-40):
        k2, v2 = ks.clone(), vs.clone()
        k2[0], v2[2] = bad, bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = _attend(new, kv, q, kc, vc, table, k2, v2, kw, status)
        assert int(status) == svw.SVW_DEV_BAD_INPUT
        assert bool(out[:, [0, 1, 4, 5]].isnan().all()) and bool(lse[:, :2].isnan().all())
        assert torch.equal(out[:, 2:4], good[0][:, 2:4]) and torch.equal(lse[:, 2:], good[1][:, 2:])


@pytest.mark.parametrize("new,kv", [([3, 1], [300, 20000]), ([150, 40], [700, 300])])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_and_queries_at_opposite_ends(new, kv, d):
    """A score is formed of factors that may be large and small; none of the steps leaves fp32's range."""
    import torch
    rng = np.random.default_rng(19)
    kc, vc, table, ks, vs = _codes(rng, new, kv, 2, d, 32)
    q = torch.zeros(sum(new), 4, d, dtype=torch.bfloat16, device="cuda")
    most = torch.full_like(ks, FLT_MAX)
    _compare_attend(new, kv, q, kc, vc, table, most, vs, {"scale": 10.0}, *_attend(new, kv, q, kc, vc, table, most, vs, {"scale": 10.0}))
    # the least scale, the largest queries
    q = _queries(rng, new, 4, d, 1).clamp(-3, 3) * 2.0 ** 125
    least = torch.full_like(ks, FLT_MIN)
    kw = {"scale": 1.3 * 2.0 ** -13 / math.sqrt(d)}
    _compare_attend(new, kv, q, kc, vc, table, least, vs, kw, *_attend(new, kv, q, kc, vc, table, least, vs, kw))


def test_a_hidden_value_beside_scales_and_queries_at_opposite_ends():
    """Rows that are formed again are formed in the same range."""
    import torch
    rng = np.random.default_rng(20)
    new, kv, d = [20], [500], 128
    kc, vc, table, ks, vs = _codes(rng, new, kv, 1, d, 16)
    q = _queries(rng, new, 2, d, 1).clamp(-3, 3) * 2.0 ** 125
    least, kw = torch.full_like(ks, FLT_MIN), {"scale": 1.3 * 2.0 ** -13 / math.sqrt(d)}
    odd = vc.clone()
    _as_bytes(odd)[int(table[0, 499 // 16]), 0, 499 % 16] = 0x7f  # the last token's values: no other sees them
    out, lse = _attend(new, kv, q, kc, odd, table, least, vs, kw)
    assert bool(out[19].isnan().all())
    clean = _attend(new, kv, q, kc, vc, table, least, vs, kw)
    out[19] = clean[0][19]
    _compare_attend(new, kv, q, kc, vc, table, least, vs, kw, out, lse)


# ---------------------------------------------------------------------------
# kv_append_norm
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("tokens", [3, 400])
@pytest.mark.parametrize("d", [64, 40])
@pytest.mark.parametrize("scale", [FLT_MIN, 1e-37, 1e-30])
def test_zeros_under_a_small_scale_are_zero(tokens, d, scale):
    """The norm's factor (1000 of a head of zeros) and a scale's reciprocal meet nowhere."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(7)
    new, kv, hkv = [tokens], [tokens], 2
    kc, vc, table = _cache(rng, new, kv, hkv, d, 16, torch.float8_e4m3fn)
    q, k, v = _append_inputs(rng, new, 2, hkv, d, torch.bfloat16)
    k, v = k.clone(), v.clone()
    k[1] = 0
    k[2, :, 1:] = 0
    v[1] = 0
    s = _f32([scale] * hkv)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    svw.kv_append_norm(k, v, kc, vc, _i32(table), _i32(_cu(new)), _i32(kv), k_weight=_f32(np.ones(d)), eps=1e-6, k_scale=s,
                       v_scale=s, status=status)
    assert int(status) == 0
    page = int(table[0, 0])
    assert bool((kc[page, :, 1].float() == 0).all()) and bool((vc[page, :, 1].float() == 0).all())
    assert bool((kc[page, :, 2, 1:].float() == 0).all()) and bool((kc[page, :, 2, 0].float().abs() == 448).all())
    assert not bool(kc[page, :, :3].float().isnan().any()) and not bool(vc[page, :, :3].float().isnan().any())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,shift", [(64, 0), (128, 0), (40, 0), (64, 1)])  # the last two: entry by entry
def test_codes_are_nearest_to_the_quotient(dtype, d, shift):
    """The nearest code to x / scale, that quotient in fp32: ties too, of which scales like 7 / 512 have many, and
    at the ends of fp32's range.  Without a norm and a rotation nothing else rounds."""
    import serving_vocab_wide_gb300 as svw
    import torch
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    scales = [7 / 512, 0.7, 1 / 3, 5 / 448, 0.03, 1.0, 2.0 ** -60, 1.1 * 2.0 ** -61, 1.9 * 2.0 ** 60, 1.7 * 2.0 ** 100,
              FLT_MIN, 1.5 * FLT_MIN, FLT_MAX, 3e38, 1.3 * 2.0 ** -100, 2.0 ** -149 * (2 ** 24 - 1)]
    hkv, page = len(scales), 16
    s = torch.tensor(scales, dtype=torch.float32)
    gen = torch.Generator().manual_seed(3)
    # per head: every bf16 number of the codes' range and beyond, of its scale; ties of fp32; anything at all
    mant = torch.arange(128, 256, dtype=torch.float64) / 128
    some = (mant[None] * 2.0 ** torch.arange(-12, 11, dtype=torch.float64)[:, None]).flatten()
    near = 2.0 ** torch.floor(torch.log2(s.double()))
    x = some[None] * near[:, None]
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    ties = (codes[1:] + codes[:-1])[None] / 2 * s.double()[:, None]
    wild = torch.randint(0, 1 << 31, (hkv, 3000), generator=gen, dtype=torch.int32).view(torch.float32).double()
    ends = torch.tensor([0.0, math.inf, math.nan, FLT_MAX, FLT_MIN, 2.0 ** -133, 2.0 ** -149], dtype=torch.float64).expand(hkv, -1)
    x = torch.cat((x, ties, wild, ends), 1).float()
    x = torch.cat((x, -x), 1).to(dt)
    tokens = -(-x.shape[1] // d)
    x = torch.nn.functional.pad(x, (0, tokens * d - x.shape[1])).view(hkv, tokens, d).transpose(0, 1).contiguous()
    want = (x.float() / s[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    store = torch.zeros(x.numel() + 1, dtype=dt, device="cuda")
    store[shift:shift + x.numel()] = x.flatten().cuda()
    y = store[shift:shift + x.numel()].view(x.shape)
    pages = -(-tokens // page)
    kc, vc = torch.zeros(2, pages, hkv, page, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    svw.kv_append_norm(y, y, kc, vc, table, _i32([0, tokens]), _i32([tokens]), k_scale=s.cuda(), v_scale=s.cuda())
    for c in (kc, vc):
        got = c.view(torch.uint8).transpose(1, 2).reshape(-1, hkv, d)[:tokens].cpu().view(torch.float8_e4m3fn).float()
        w = want.float()
        same = (got == w) | (got.isnan() & w.isnan())
        assert bool(same.all()), [(float(x[tuple(i)]), scales[int(i[1])], float(got[tuple(i)]), float(w[tuple(i)]))
                                  for i in (~same).nonzero()[:5]] + [int((~same).sum())]


@pytest.mark.parametrize("codes,weight", [(False, False), (False, True), (True, False), (True, True)])
def test_the_timer_of_its_name_fires(codes, weight):
    """Whatever kernel serves a call, a timer armed for kv_append_norm records around it."""
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(8)
    kc, vc, table = _cache(rng, [5], [5], 2, 64, 16, torch.float8_e4m3fn if codes else torch.bfloat16)
    q, k, v = _append_inputs(rng, [5], 2, 2, 64, torch.bfloat16)
    start, begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(3))
    start.record()
    svw.time_next_launch("kv_append_norm", begin, end)
    torch.cuda._sleep(20_000_000)  # some 10 ms
    svw.kv_append_norm(k, v, kc, vc, _i32(table), _i32([0, 5]), _i32([5]), k_weight=_f32(np.ones(64)) if weight else None)
    torch.cuda.synchronize()
    svw.time_next_launch(None)
    assert start.elapsed_time(begin) > 2 and begin.elapsed_time(end) > 0


# ---------------------------------------------------------------------------
# kv_gather
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("cache", ["e4m3", "bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 24])
def test_one_side_alone(cache, d):
    import serving_vocab_wide_gb300 as svw
    import torch
    rng = np.random.default_rng(4)
    dt = {"e4m3": torch.float8_e4m3fn, "bf16": torch.bfloat16, "fp32": torch.float32}[cache]
    n = [20, 7]
    kc, vc, table = _cache(rng, n, n, 2, d, 16, dt)
    args = kc, vc, _i32(table), _i32(_cu(n))
    both = svw.kv_gather(*args)
    k, none = svw.kv_gather(*args, want_v=False)
    assert none is None and torch.equal(k, both[0])
    given = torch.empty(27, 2, d, device="cuda")
    none, v = svw.kv_gather(*args, want_k=False, v_out=given)
    assert none is None and v is given and torch.equal(v.bfloat16(), both[1])
