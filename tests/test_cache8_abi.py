"""Host-side validation of the calls of an 8-bit cache (kv_append_norm,
kv_gather, paged_attention_fp8) through the C ABI and in Python, without a GPU."""
import ctypes

import pytest
import torch

from test_round_abi import INVALID, MISALIGNED, OK, P, UNSUPPORTED, WORKSPACE, _kv, svw  # noqa: F401 (a fixture)
from test_round_host import BF16, F32, I32, U8, Stream, Tensor, host  # noqa: F401 (a fixture)

F8 = torch.float8_e4m3fn


def _append(svw, cache=None, **o):
    a = dict(k=P, kt=256, kh=64, v=P, vt=256, vh=64, q=P, qt=256, qh=64, qo=P + 0x10000, dt=1, hq=4, N=2, cu=P, T=5,
             kv=P, pos=None, kw=P, qw=P, eps=1e-6, cs=P, maxpos=100, rot=64, inter=0)
    b = dict(cdt=2, ks=P, vs=P)
    for k, v in o.items():
        (a if k in a else b)[k] = v
    c = _kv(svw) if cache is None else cache
    return svw.lib().kv_append_norm(*a.values(), ctypes.byref(c) if c else None, *b.values(), P, None)


@pytest.mark.parametrize("o,want", [
    ({"dt": 3}, UNSUPPORTED), ({"dt": 2}, UNSUPPORTED), ({"cdt": 0}, UNSUPPORTED), ({"cdt": 3}, UNSUPPORTED),
    ({"dt": 0, "cdt": 1}, UNSUPPORTED), ({"N": 0}, INVALID), ({"T": -1}, INVALID), ({"k": None}, INVALID),
    ({"cu": None}, INVALID), ({"qo": None}, INVALID), ({"q": None}, INVALID), ({"q": None, "qo": None}, INVALID),
    ({"hq": 0}, INVALID), ({"rot": 63}, INVALID), ({"rot": 66}, INVALID), ({"cs": None}, INVALID), ({"kt": -1}, INVALID),
    ({"eps": -1e-6}, INVALID), ({"eps": float("nan")}, INVALID), ({"eps": float("inf")}, INVALID),
    ({"cdt": 1}, INVALID), ({"k": P + 1}, MISALIGNED), ({"kw": P + 2}, MISALIGNED), ({"qw": P + 1}, MISALIGNED),
    ({"ks": P + 2}, MISALIGNED), ({"vs": P + 1}, MISALIGNED), ({"qo": P, "qt": 512}, INVALID), ({"T": 0}, OK),
    ({"T": 0, "cdt": 1, "ks": None, "vs": None}, OK)])
def test_append_norm_validates(svw, o, want):  # noqa: F811
    assert _append(svw, **o) == want


@pytest.mark.parametrize("f,cdt,want", [
    ({"k": None}, 2, INVALID), ({"n_pages": 0}, 2, INVALID), ({"table_stride": 7}, 2, INVALID),
    ({"k_stride": (-1, 64, 64)}, 2, INVALID), ({"head_dim": 2048}, 2, UNSUPPORTED), ({"k": P + 1}, 1, MISALIGNED)])
def test_append_norm_validates_the_cache(svw, f, cdt, want):  # noqa: F811
    scales = {} if cdt == 2 else {"ks": None, "vs": None}
    assert _append(svw, cache=_kv(svw, **f), cdt=cdt, **scales) == want


def _gather(svw, cache=None, **o):
    a = dict(cdt=2, ks=P, vs=P, N=2, cu=P, T=5, first=P, ko=P, vo=P, odt=1, st=P, stream=None)
    a.update(o)
    c = _kv(svw) if cache is None else cache
    return svw.lib().kv_gather(ctypes.byref(c) if c else None, *a.values())


@pytest.mark.parametrize("o,want", [
    ({"cdt": 3}, UNSUPPORTED), ({"odt": 2}, UNSUPPORTED), ({"N": 0}, INVALID), ({"T": -1}, INVALID),
    ({"T": 1 << 31}, UNSUPPORTED), ({"cu": None}, INVALID), ({"ko": None, "vo": None}, INVALID), ({"cdt": 1}, INVALID),
    ({"ko": P + 1}, MISALIGNED), ({"first": P + 2}, MISALIGNED), ({"cu": P + 1}, MISALIGNED), ({"ks": P + 1}, MISALIGNED),
    ({"T": 0}, OK), ({"T": 0, "ko": None, "vo": None}, OK)])
def test_gather_validates(svw, o, want):  # noqa: F811
    assert _gather(svw, **o) == want


def test_gather_validates_the_cache(svw):  # noqa: F811
    assert _gather(svw, cache=_kv(svw, n_pages=0)) == INVALID
    assert _gather(svw, cache=_kv(svw, head_dim=1025)) == UNSUPPORTED
    assert _gather(svw, cache=_kv(svw, v=P + 2), cdt=0, ks=None, vs=None) == MISALIGNED
    assert svw.lib().kv_gather(None, 2, None, None, 1, P, 1, None, P, P, 1, None, None) == INVALID


def _attend(svw, cache=None, **o):
    a = dict(q=P, qt=256, qh=64, dt=1, hq=4, N=2, cu=P, T=5, kv=P)
    b = dict(ks=P, vs=P, scale=0.1, causal=1, window=0, out=P, lse=P, st=P, ws=P, wb=1 << 40, stream=None)
    for k, v in o.items():
        (a if k in a else b)[k] = v
    c = _kv(svw) if cache is None else cache
    return svw.lib().paged_attention_fp8(*a.values(), ctypes.byref(c), *b.values())


@pytest.mark.parametrize("o,want", [
    ({"dt": 0}, UNSUPPORTED), ({"dt": 2}, UNSUPPORTED), ({"N": 0}, INVALID), ({"hq": 5}, INVALID),
    ({"hq": 130}, UNSUPPORTED), ({"q": None}, INVALID), ({"out": None}, INVALID), ({"scale": 0.0}, INVALID),
    ({"scale": float("nan")}, INVALID), ({"window": -1}, INVALID), ({"window": 3, "causal": 0}, INVALID),
    ({"q": P + 8}, MISALIGNED), ({"qt": 260}, MISALIGNED), ({"ks": P + 2}, MISALIGNED), ({"vs": P + 1}, MISALIGNED),
    ({"qh": 0}, UNSUPPORTED), ({"ws": P + 16}, MISALIGNED), ({"ws": None}, WORKSPACE), ({"wb": 0}, WORKSPACE),
    ({"T": 0}, OK)])
def test_attend_fp8_validates(svw, o, want):  # noqa: F811
    assert _attend(svw, **o) == want


@pytest.mark.parametrize("f,want", [
    ({"page_size": 8}, UNSUPPORTED), ({"page_size": 24}, UNSUPPORTED), ({"head_dim": 96}, UNSUPPORTED),
    ({"k_stride": (2048, 1024, 72)}, MISALIGNED), ({"v": P + 8}, MISALIGNED), ({"v_stride": (0, 1024, 64)}, UNSUPPORTED)])
def test_attend_fp8_validates_the_cache(svw, f, want):  # noqa: F811
    assert _attend(svw, cache=_kv(svw, **f)) == want


# ---------------------------------------------------------------------------
# the Python calls, with stand-ins for the GPU's tensors and streams
# ---------------------------------------------------------------------------
@pytest.fixture
def calls(host, monkeypatch):  # noqa: F811
    """The calls of an 8-bit cache recorded, as test_round_host's are."""
    import serving_vocab_wide_gb300 as m
    before = m.lib()

    class Lib:
        def __getattr__(self, name):
            if name in ("kv_append_norm", "kv_gather", "paged_attention_fp8"):
                return lambda *a: host.calls.append((name, a)) or 0
            return getattr(before, name)

    monkeypatch.setattr(m, "lib", lambda: Lib())
    m._torch().float8_e4m3fn = F8

    def make(gpu=0, **kw):
        t = lambda shape, dtype: Tensor(shape, dtype, gpu=gpu)
        paged = (t((10, 2, 16, 64), F8), t((10, 2, 16, 64), F8), t((3, 4), I32), t((4,), I32))
        scales = {"k_scale": t((2,), F32), "v_scale": t((2,), F32)}
        q, k, v = t((9, 4, 64), BF16), t((9, 2, 64), BF16), t((9, 2, 64), BF16)
        return {
            "paged_attention_fp8": lambda **o: m.paged_attention_fp8(q, *paged, t((3,), I32), **{**scales, **kw, **o}),
            "kv_append_norm": lambda **o: m.kv_append_norm(
                k, v, *paged, t((3,), I32), **{"q": q, "k_weight": t((64,), F32), "q_weight": t((64,), F32), **scales,
                                              **kw, **o}),
            "kv_gather": lambda **o: m.kv_gather(*paged, **{"total_out": 9, **scales, **kw, **o}),
        }
    return host, make


@pytest.mark.parametrize("name,outputs,workspaces", [("paged_attention_fp8", 2, 1), ("kv_append_norm", 1, 0), ("kv_gather", 2, 0)])
def test_memory_comes_from_the_stream_that_uses_it(calls, name, outputs, workspaces):
    h, make = calls
    side, current = Stream(9), h.current
    make(stream=side)[name]()
    assert len(h.made) == outputs + workspaces and h.current is current
    assert all(t.pool is side for t in h.made)
    assert h.calls[0][0] == name and h.calls[0][1][-1] == side.cuda_stream
    assert [t.dtype for t in h.made].count(U8) == workspaces
    for t in h.made:
        assert t.recorded == ([] if t.dtype is U8 else [current])


@pytest.mark.parametrize("name", ["paged_attention_fp8", "kv_append_norm", "kv_gather"])
def test_another_gpu_than_the_current_one_is_refused(calls, name):
    import serving_vocab_wide_gb300 as m
    h, make = calls
    h.device = 1
    with pytest.raises(m.SvwError, match="current"):
        make()[name]()
    h.device = 0
    with pytest.raises(m.SvwError, match="current"):
        make(stream=Stream(9, gpu=1))[name]()
    with pytest.raises(m.SvwError):
        make()[name](k_scale=Tensor((2,), F32, gpu=1))
    assert not h.made and not h.calls


@pytest.mark.parametrize("name,o", [
    ("kv_append_norm", {"k_scale": Tensor((3,), F32)}), ("kv_append_norm", {"v_scale": Tensor((2,), BF16)}),
    ("kv_append_norm", {"k_weight": Tensor((63,), F32)}), ("kv_append_norm", {"q_weight": Tensor((64,), BF16)}),
    ("kv_append_norm", {"q": None}), ("kv_append_norm", {"q": None, "q_weight": None, "q_out": Tensor((9, 4, 64), BF16)}),
    ("kv_append_norm", {"positions": Tensor((8,), I32)}), ("kv_append_norm", {"q_out": Tensor((9, 4, 64), F32)}),
    ("kv_gather", {"first": Tensor((4,), I32)}), ("kv_gather", {"dtype": torch.float16}), ("kv_gather", {"dtype": F8}),
    ("kv_gather", {"k_out": Tensor((8, 2, 64), BF16)}), ("kv_gather", {"dtype": BF16, "v_out": Tensor((9, 2, 64), F32)}),
    ("kv_gather", {"k_scale": Tensor((1,), F32)}), ("paged_attention_fp8", {"v_scale": Tensor((4,), F32)}),
    ("paged_attention_fp8", {"out": Tensor((9, 4, 64), F32)}), ("paged_attention_fp8", {"lse": Tensor((35,), F32)}),
    ("paged_attention_fp8", {"workspace": Tensor((1 << 20,), F32)})])
def test_refusals(calls, name, o):
    import serving_vocab_wide_gb300 as m
    h, make = calls
    make()[name]()
    with pytest.raises(m.SvwError):
        make()[name](**o)
    assert len(h.calls) == 1


def test_scales_come_with_codes(calls):
    """Caches of another type have no scales, and take tokens of their own type only."""
    import serving_vocab_wide_gb300 as m
    h, _ = calls
    t = Tensor
    where = (t((10, 2, 16, 64), BF16), t((10, 2, 16, 64), BF16), t((3, 4), I32), t((4,), I32))
    k, v, n, s = t((9, 2, 64), BF16), t((9, 2, 64), BF16), t((3,), I32), t((2,), F32)
    m.kv_append_norm(k, v, *where, n)
    m.kv_gather(*where, total_out=9, dtype=F32)
    for call in (lambda: m.kv_append_norm(k, v, *where, n, k_scale=s), lambda: m.kv_gather(*where, total_out=9, v_scale=s),
                 lambda: m.kv_append_norm(t((9, 2, 64), F32), t((9, 2, 64), F32), *where, n),
                 lambda: m.paged_attention_fp8(t((9, 4, 64), BF16), *where, n)):
        with pytest.raises(m.SvwError):
            call()
    assert len(h.calls) == 2


def test_gather_of_one_side(calls):
    """No memory is taken, and no address handed over, for the side that is not wanted."""
    import serving_vocab_wide_gb300 as m
    h, make = calls
    gather = make()["kv_gather"]
    k, v = gather(want_v=False)
    assert v is None and k.shape == (9, 2, 64) and len(h.made) == 1
    assert h.calls[-1][1][8] == 0x10000 and h.calls[-1][1][9] == 0
    given = Tensor((9, 2, 64), F32)
    assert gather(want_k=False, v_out=given) == (None, given) and len(h.made) == 1
    assert h.calls[-1][1][8] == 0 and h.calls[-1][1][9] == 0x10000
    for o in ({"want_k": False, "want_v": False}, {"want_k": False, "k_out": given}, {"want_v": False, "v_out": given}):
        with pytest.raises(m.SvwError):
            gather(**o)
    assert len(h.calls) == 2
