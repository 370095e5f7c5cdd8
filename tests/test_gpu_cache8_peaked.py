"""paged_attention_fp8 on rows with one key far above a long tail of others (a
first token, a copied one): the tail's weights are small, but together they are
a part of the output."""
import numpy as np
import pytest

import cache8_reference as c8
import round_reference as ref
from test_gpu_cache8 import _check_attend, _codes, _queries
from test_gpu_paged import ATTEND, _cu, _i32, _lib  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def _cache_of(gen, keys, hkv, d, page, first, one):
    """Codes of `keys` tokens (the pages in a shuffled order): key element 0 is 1 at token `first` and 0
    elsewhere, element 1 unit normal, values about 1 (the first's small), or all of them 1."""
    import torch
    k = torch.zeros(hkv, keys, d, device="cuda")
    k[:, :, 1] = torch.randn(hkv, keys, generator=gen, device="cuda")
    k[:, first, :2] = torch.tensor([1.0, 0.0], device="cuda")
    v = 1 + 0.25 * torch.randn(hkv, keys, d, generator=gen, device="cuda")
    v[:, first] = 0.0625 * torch.randn(hkv, d, generator=gen, device="cuda")
    if one:
        v[:] = 1
    k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
    pages = -(-keys // page)
    table = torch.randperm(pages, generator=gen, device="cuda").int()
    caches = []
    for x in (k, v):
        c = torch.zeros(pages, hkv, page, d, dtype=torch.uint8, device="cuda")
        full = torch.zeros(hkv, pages * page, d, dtype=torch.uint8, device="cuda")
        full[:, :keys] = x.view(torch.uint8)
        c[table.long()] = full.view(hkv, pages, page, d).transpose(0, 1)
        caches.append(c.view(torch.float8_e4m3fn))
    return k.double(), v.double(), caches, table


FORMS = [
    ([1], 8, 2, 128), ([1], 2, 2, 64), ([17], 4, 1, 128),        # narrow, keys of a unit on many workers
    ([1] * 64, 16, 8, 128), ([3] * 64, 16, 8, 64),               # narrow, a unit on one worker
    ([300], 2, 1, 128), ([300], 2, 1, 64), ([150] * 48, 4, 4, 128),  # wide
]


@pytest.mark.parametrize("nats,keys", [(8, 2000), (11, 2000), (11, 8001), (11, 16000), (14, 16000), (12, 131072), (14, 131072),
                                       (16, 131072)])
@pytest.mark.parametrize("spread", [0.0, 0.5])
@pytest.mark.parametrize("new,hq,hkv,d", FORMS)
def test_a_far_maximum_leaves_the_tail(new, hq, hkv, d, nats, keys, spread):
    """Bound, for up to 2^17 keys: the output's rounding, and 2^-8 of the weighted
    magnitudes: weights' rounding (2^-11), scores and exponentials (2^-10.7), the
    two sums in fp32 (2^-11 and 2^-9)."""
    import serving_vocab_wide_gb300 as svw
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(keys + nats + d)
    one = spread == 0.0 and nats % 2 == 1
    first = 0 if nats < 14 else keys // 3
    k, v, caches, table = _cache_of(gen, keys, hkv, d, 64, first, one)
    n, t = len(new), sum(new)
    q = torch.zeros(t, hq, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = nats
    q[..., 1] = spread * (1 + torch.randint(0, 2, (t, hq), generator=gen, device="cuda"))
    kv = [keys] * n
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = svw.paged_attention_fp8(q, *caches, table[None].expand(n, -1).contiguous(), _i32(_cu(new)), _i32(kv), scale=1.0,
                                       status=status)
    assert int(status) == 0
    # all requests see the same keys, up to their own
    last = torch.cat([torch.arange(keys - m, keys, device="cuda") for m in new])
    j = torch.arange(keys, device="cuda")
    for h in (0, hq - 1):
        for rows in torch.arange(t, device="cuda").split(64):
            if t > 1000 and int(rows[0]) % 1024:
                continue
            hk = h // (hq // hkv)
            x = q[rows, h].double() @ k[hk].T
            x = x.masked_fill(j[None] > last[rows, None], -torch.inf)
            want_lse = torch.logsumexp(x, 1)
            w = torch.exp(x - want_lse[:, None])
            want, mass = w @ v[hk], w @ v[hk].abs()
            err = (out[rows, h].double() - want).abs()
            bound = 2.0 ** -8 * mass + 1.01 * 2.0 ** -8 * want.abs()
            assert bool((err <= bound).all()), f"{float((err / bound).max())} of the bound"
            assert bool(((lse[rows, h].double() - want_lse).abs() <= 1e-3).all())


def test_the_same_row_alone_and_in_a_batch():
    """A row's keys cut into many parts or into none: the same output but for
    roundings (two of its own, and 2^-9 of the weighted magnitudes for each)."""
    import serving_vocab_wide_gb300 as svw
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    keys, hq, hkv, d = 16000, 16, 8, 128
    _, _, caches, table = _cache_of(gen, keys, hkv, d, 64, 0, False)
    q = torch.zeros(64, hq, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 11
    q[..., 1] = 0.5
    many, _ = svw.paged_attention_fp8(q, *caches, table[None].expand(64, -1).contiguous(), _i32(range(65)), _i32([keys] * 64), scale=1.0)
    one, _ = svw.paged_attention_fp8(q[:1], *caches, table[None].contiguous(), _i32([0, 1]), _i32([keys]), scale=1.0)
    # the outputs are averages of values of 2 at most: a mass of 2 bounds them
    assert float((many[:1].float() - one.float()).abs().max()) <= 2 * (2.0 ** -8 * 2 + 2.0 ** -9 * 2)


@pytest.mark.parametrize("new", [[1], [300]])
@pytest.mark.parametrize("d", [64, 128])
def test_every_code_as_a_value(new, d):
    """Each finite code alone, the least ones too: equal scores of one key leave it as it is."""
    import serving_vocab_wide_gb300 as svw
    import torch
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    codes = codes[(codes & 0x7f) != 0x7f].view(torch.float8_e4m3fn)  # 254 of them: one for each request and element
    n = 254
    v = codes.view(torch.uint8)[(torch.arange(n, device="cuda")[:, None] + torch.arange(d, device="cuda")[None]) % n]
    vc = torch.zeros(n, 1, 16, d, dtype=torch.uint8, device="cuda")
    vc[:, 0, 0] = v
    vc[:, 0, 1:] = 0x7f  # beyond the request's one key
    kc = torch.zeros(n, 1, 16, d, dtype=torch.float8_e4m3fn, device="cuda")
    t = n * new[0]
    q = torch.ones(t, 1, d, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous()
    out, lse = svw.paged_attention_fp8(q, kc, vc.view(torch.float8_e4m3fn), table, _i32(np.arange(n + 1) * new[0]), _i32([1] * n),
                                       causal=False)
    want = v.view(torch.float8_e4m3fn).float()[:, None].expand(n, new[0], d).reshape(t, 1, d)
    assert torch.equal(out.float(), want) and float(lse.abs().max()) == 0


def _attend_closely(q, k, v, scale, causal, window):
    """round_reference's attend; its bounds, which hold weights of eight bits, widened by the queries' two numbers alone."""
    out, lse, ob, lb = ref.attend(q, k, v, scale, causal, window)
    most = np.abs(q).max(1, keepdims=True)
    q_err = np.where(np.abs(q) < 2.0 ** -9 * most, 2.0 ** -17 * most, 0.0)
    n, kv = q.shape[0], k.shape[0]
    at, j = kv - n + np.arange(n)[:, None], np.arange(kv)[None]
    ok = (j <= at) & (j > at - (window or kv + n)) if causal else np.ones((n, kv), bool)
    eps = (scale * (q_err @ np.abs(k).T) * ok).max(1, initial=0.0)
    w = np.where(ok, np.exp(np.minimum(scale * (q @ k.T) - np.where(np.isfinite(lse), lse, 0)[:, None], 0)), 0.0)
    return out, lse, ob + 2 * eps[:, None] * (w @ np.abs(v)), lb + 2 * eps


@pytest.mark.parametrize("new,kv,hq,hkv,d,page,tf,kw", ATTEND)
def test_parity_without_a_term_of_all_keys(new, kv, hq, hkv, d, page, tf, kw, monkeypatch):
    monkeypatch.setattr(c8, "attend", _attend_closely)
    rng = np.random.default_rng(sum(kv) + hq + 1)
    kc, vc, table, ks, vs = _codes(rng, new, kv, hkv, d, page, tf)
    _check_attend(new, kv, _queries(rng, new, hq, d), kc, vc, table, ks, vs, kw)
