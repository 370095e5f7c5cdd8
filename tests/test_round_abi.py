"""Host-side validation of the round's calls (logits_adjust, kv_append,
paged_attention) through the C ABI, without a GPU."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
P = 0x10000  # any aligned non-null pointer: a refused call never reads it


@pytest.fixture(scope="module")
def svw():
    import serving_vocab_wide_gb300 as m
    m.build()
    m.lib()
    return m


def _adjust(svw, **o):
    a = dict(logits=P, ls=100, dt=1, V=100, N=2, cu=P, R=3, bonus=1, tok=P, hist=P, cuh=P, nh=5, pl=P, rep=P, freq=P,
             pres=P, bt=P, bv=P, cub=P, nb=2, mask=P, mr=4, mrow=P, out=P + 0x10000, os=100, st=P, ws=None, wb=0, stream=None)
    a.update(o)
    return svw.lib().logits_adjust(*a.values())


@pytest.mark.parametrize("o,want", [
    ({"dt": 2}, UNSUPPORTED), ({"V": 0}, INVALID), ({"N": 0}, INVALID), ({"R": -1}, INVALID), ({"V": 1 << 21}, UNSUPPORTED),
    ({"nh": 1 << 31}, UNSUPPORTED), ({"logits": None}, INVALID), ({"out": None}, INVALID), ({"cu": None}, INVALID),
    ({"tok": None}, INVALID), ({"hist": None}, INVALID), ({"bv": None}, INVALID), ({"ls": 99}, INVALID),
    ({"os": 99}, INVALID), ({"mrow": None}, INVALID), ({"logits": P + 1}, MISALIGNED), ({"cu": P + 2}, MISALIGNED),
    ({"mask": P + 2}, MISALIGNED), ({"out": P + 64}, INVALID), ({"out": P, "os": 104}, INVALID),
    ({"ws": P + 16}, MISALIGNED), ({"N": 500, "V": 65536, "ls": 65536, "os": 65536, "mr": 503, "ws": P, "wb": 256}, WORKSPACE),
    ({"R": 0, "tok": None, "bonus": 0, "mask": None}, OK)])
def test_adjust_validates(svw, o, want):
    assert _adjust(svw, **o) == want


def _kv(svw, **o):
    f = dict(k=P, v=P, k_stride=(2048, 1024, 64), v_stride=(2048, 1024, 64), block_table=P, table_stride=8, max_pages=8,
             n_pages=10, page_size=16, n_kv_heads=2, head_dim=64)
    f.update(o)
    return svw._PagedKV(*f.values())


def _append(svw, cache=None, **o):
    a = dict(k=P, kt=256, kh=64, v=P, vt=256, vh=64, q=P, qt=256, qh=64, qo=P + 0x10000, dt=1, hq=4, N=2, cu=P, T=5,
             kv=P, pos=None, cs=P, maxpos=100, rot=64, inter=0)
    a.update(o)
    c = _kv(svw) if cache is None else cache
    return svw.lib().kv_append(*a.values(), ctypes.byref(c) if c else None, P, None)


@pytest.mark.parametrize("o,want", [
    ({"dt": 3}, UNSUPPORTED), ({"N": 0}, INVALID), ({"T": -1}, INVALID), ({"k": None}, INVALID), ({"cu": None}, INVALID),
    ({"qo": None}, INVALID), ({"q": None}, INVALID), ({"hq": 0}, INVALID), ({"rot": 63}, INVALID), ({"rot": 66}, INVALID),
    ({"cs": None}, INVALID), ({"maxpos": 0}, INVALID), ({"kt": -1}, INVALID), ({"k": P + 1}, MISALIGNED),
    ({"cs": P + 1}, MISALIGNED), ({"qo": P, "qt": 512}, INVALID), ({"T": 0}, OK)])
def test_append_validates(svw, o, want):
    assert _append(svw, **o) == want


@pytest.mark.parametrize("f,want", [
    ({"k": None}, INVALID), ({"block_table": None}, INVALID), ({"n_pages": 0}, INVALID), ({"page_size": 0}, INVALID),
    ({"table_stride": 7}, INVALID), ({"k_stride": (-1, 64, 64)}, INVALID), ({"head_dim": 2048}, UNSUPPORTED),
    ({"block_table": P + 1}, MISALIGNED)])
def test_append_validates_the_cache(svw, f, want):
    assert _append(svw, cache=_kv(svw, **f)) == want


def test_null_cache(svw):
    L = svw.lib()
    assert L.kv_append(P, 1, 1, P, 1, 1, None, 0, 0, None, 1, 0, 1, P, 1, P, None, None, 0, 0, 0, None, None, None) == INVALID
    assert L.paged_attention(P, 64, 64, 1, 4, 1, P, 1, P, None, 1.0, 1, 0, P, None, None, P, 1 << 30, None) == INVALID


def _attend(svw, cache=None, **o):
    a = dict(q=P, qt=256, qh=64, dt=1, hq=4, N=2, cu=P, T=5, kv=P)
    b = dict(scale=0.1, causal=1, window=0, out=P, lse=P, st=P, ws=P, wb=1 << 40, stream=None)
    for k, v in o.items():
        (a if k in a else b)[k] = v
    c = _kv(svw) if cache is None else cache
    return svw.lib().paged_attention(*a.values(), ctypes.byref(c), *b.values())


@pytest.mark.parametrize("o,want", [
    ({"dt": 0}, UNSUPPORTED), ({"N": 0}, INVALID), ({"hq": 5}, INVALID), ({"hq": 130}, UNSUPPORTED), ({"q": None}, INVALID),
    ({"out": None}, INVALID), ({"scale": 0.0}, INVALID), ({"scale": float("nan")}, INVALID), ({"window": -1}, INVALID),
    ({"window": 3, "causal": 0}, INVALID), ({"q": P + 8}, MISALIGNED), ({"qt": 260}, MISALIGNED), ({"qh": 0}, UNSUPPORTED),
    ({"ws": P + 16}, MISALIGNED), ({"ws": None}, WORKSPACE), ({"wb": 0}, WORKSPACE), ({"T": 0}, OK)])
def test_attend_validates(svw, o, want):
    assert _attend(svw, **o) == want


@pytest.mark.parametrize("f,want", [
    ({"page_size": 8}, UNSUPPORTED), ({"page_size": 24}, UNSUPPORTED), ({"page_size": 2048}, UNSUPPORTED),
    ({"head_dim": 96}, UNSUPPORTED), ({"k_stride": (2048, 1024, 60)}, MISALIGNED), ({"v": P + 2}, MISALIGNED),
    ({"v_stride": (0, 1024, 64)}, UNSUPPORTED)])
def test_attend_validates_the_cache(svw, f, want):
    assert _attend(svw, cache=_kv(svw, **f)) == want


def test_attention_workspace_size(svw):
    f = svw.paged_attention_workspace_size
    assert f(10, 8, 2, 128) > 0 and f(10, 8, 2, 128) % 256 == 0
    assert f(10, 7, 2, 128) == 0 and f(10, 8, 2, 96) == 0 and f(-1, 8, 2, 128) == 0 and f(10, 130, 2, 128) == 0


def test_adjust_workspace_size(svw):
    f = svw.logits_adjust_workspace_size
    assert f(1, 32000, 0, 64, 0) == 0          # a small batch counts for itself
    assert f(1, 32000, 0, 1 << 17, 0) > (16 << 17)  # a long history does not
    n = f(256, 151936, 2000, 500000, 8192)
    assert n >= 16 * (2000 + 500000 + 8192) and n % 256 == 0
    assert f(0, 100, 0, 0, 0) == 0 and f(1, 1 << 21, 0, 0, 0) == 0 and f(1, 100, -1, 0, 0) == 0
