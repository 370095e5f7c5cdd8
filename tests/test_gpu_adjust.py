"""GPU parity of logits_adjust against its definition in 64 bits."""
import numpy as np
import pytest

import round_reference as ref

pytestmark = pytest.mark.gpu
NEG = -3.3895314e38  # the lowest finite bf16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    import serving_vocab_wide_gb300 as svw
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    svw.build()
    svw.lib()


def _case(seed, lens, V, dtype, hist=(0, 200), nbias=5, masked=True, bonus=True):
    import torch
    rng = np.random.default_rng(seed)
    N, R = len(lens), int(np.sum(lens))
    rows = R + (N if bonus else 0)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    x = rng.normal(0, 3, (rows, V)).astype(np.float32)
    few = rng.integers(0, V, min(V, 20))
    pick = lambda n: np.where(rng.random(n) < 0.7, rng.choice(few, n), rng.integers(0, V, n)).astype(np.int32)
    hl = rng.integers(hist[0], hist[1] + 1, N)
    cu_h = np.concatenate([[0], np.cumsum(hl)]).astype(np.int32)
    # values a model or an earlier step may leave: banned, overflowed, at the type's end
    for val in (-np.inf, np.inf, NEG, 0.0):
        x[rng.integers(0, rows, 8), rng.choice(few, 8)] = val
    t = torch.from_numpy(x)
    if dtype == "bf16":
        t = t.to(torch.bfloat16)
    c = {"x": t.double().numpy(), "t": t, "cu": cu, "tokens": pick(R), "history": pick(int(hl.sum())), "cu_h": cu_h,
         "prompt": np.array([rng.integers(0, h + 1) for h in hl], np.int32),
         "rep": rng.uniform(0.5, 1.8, N).astype(np.float32), "freq": rng.uniform(-0.5, 1, N).astype(np.float32),
         "pres": rng.uniform(-0.5, 1, N).astype(np.float32), "bonus": bonus, "V": V, "rows": rows}
    # a token may be listed twice: the last one counts
    c["biases"] = [[(int(v), float(np.float32(b))) for v, b in
                    zip(rng.choice(few, nbias), rng.choice([-np.inf, 1.5, -2.25, 7.0], nbias))] for _ in range(N)]
    c["mask"] = c["mask_row"] = None
    if masked:
        m = rng.random((4, V)) < np.array([0.02, 0.5, 0.98, 0.0])[:, None]  # the last row allows nothing
        c["mask"], c["mask_row"] = m, rng.integers(-1, 4, rows).astype(np.int32)
        c["mask_row"][0] = 3
    return c


def _words(mask):
    V = mask.shape[1]
    W = (V + 31) // 32
    bits = np.ones((mask.shape[0], W * 32), np.uint64)  # bits beyond V mean nothing
    bits[:, :V] = mask
    words = (bits.reshape(-1, W, 32) << np.arange(32, dtype=np.uint64)).sum(2)
    return words.astype(np.uint32).view(np.int32)


def _args(c, **over):
    import torch
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    N = len(c["cu"]) - 1
    kw = {"history": d(c["history"]), "cu_history": d(c["cu_h"]), "prompt_len": d(c["prompt"]),
          "repetition": d(c["rep"]), "frequency": d(c["freq"]), "presence": d(c["pres"]),
          "has_bonus": c["bonus"], "total_draft_rows": int(c["cu"][-1])}
    if any(c["biases"]):
        flat = [e for b in c["biases"] for e in b]
        kw["bias_tokens"] = d(np.array([v for v, _ in flat], np.int32))
        kw["bias_values"] = d(np.array([b for _, b in flat], np.float32))
        kw["cu_bias"] = d(np.cumsum([0] + [len(b) for b in c["biases"]]).astype(np.int32))
    if c["mask"] is not None:
        kw["mask"], kw["mask_row"] = d(_words(c["mask"])), d(c["mask_row"])
    kw.update(over)
    return (d(c["cu"]), d(c["tokens"])), kw


def _reference(c):
    return ref.adjust(c["x"], c["cu"], c["tokens"], c["history"], c["cu_h"], c["prompt"], c["rep"].astype(float),
                      c["freq"].astype(float), c["pres"].astype(float), c["biases"], c["mask"], c["mask_row"],
                      c["bonus"])


def _compare(got, c, reference=None, rows=slice(None)):
    import torch
    y, size = _reference(c) if reference is None else reference
    y, size = y[rows], size[rows]
    bf16 = c["t"].dtype == torch.bfloat16
    g = got.double().cpu().numpy()[rows]
    top = 3.3961775e38 if bf16 else 3.4028235e38  # beyond: rounds to infinity
    with np.errstate(invalid="ignore"):
        y = np.where(np.abs(y) > top, np.sign(y) * np.inf, y)
    assert np.array_equal(np.isnan(g), np.isnan(y))
    assert np.array_equal(np.isinf(g), np.isinf(y)) and np.array_equal(g[np.isinf(y)], y[np.isinf(y)])
    fine = np.isfinite(y)
    err = np.abs(g - y)[fine]
    bound = ref.adjust_bound(y, size, bf16)[fine]
    assert np.all(err <= bound), f"worst {np.max(err / np.maximum(bound, 1e-300))} of the bound"


SHAPES = [([0], 40, "bf16"), ([1], 1, "fp32"), ([3, 0, 16, 1], 1000, "bf16"), ([3, 0, 16, 1], 1001, "bf16"),
          ([2, 5], 5003, "fp32"), ([32, 32], 8192, "fp32"), ([4] * 9, 32001, "bf16"), ([16, 2, 8], 151936, "bf16"),
          ([1] * 40, 4104, "bf16"), ([7], 70000, "fp32"),
          # more requests; then enough that their lists are counted first
          ([3, 0] * 23, 32001, "bf16"), ([2] * 64, 20488, "fp32"), ([1] * 310, 300, "bf16"),
          ([3, 0] * 64, 32001, "bf16"), ([2] * 150, 20488, "fp32"), ([1] * 1200, 300, "bf16")]


@pytest.mark.parametrize("lens,V,dtype", SHAPES)
@pytest.mark.parametrize("bonus", [True, False])
def test_adjust_parity(lens, V, dtype, bonus):
    import serving_vocab_wide_gb300 as svw
    if not bonus and sum(lens) == 0:
        lens = [2]
    c = _case(11 + V, lens, V, dtype, bonus=bonus)
    a, kw = _args(c)
    out = svw.logits_adjust(c["t"].cuda(), *a, **kw)
    _compare(out, c)
    again = svw.logits_adjust(c["t"].cuda(), *a, **kw)
    import torch
    ints = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(out.view(ints), again.view(ints))


@pytest.mark.parametrize("lens,V,dtype", SHAPES)
def test_adjust_in_place(lens, V, dtype):
    import serving_vocab_wide_gb300 as svw
    import torch
    c = _case(5 + V, lens, V, dtype)
    a, kw = _args(c)
    x = c["t"].cuda()
    apart = svw.logits_adjust(x, *a, **kw)
    y = svw.logits_adjust(x, *a, out=x, **kw)
    assert y.data_ptr() == x.data_ptr()
    ints = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(apart.view(ints), x.view(ints))
    _compare(x, c)


@pytest.mark.parametrize("drop", ["history", "bias", "mask", "factors", "all"])
def test_adjust_parts_left_out(drop):
    import serving_vocab_wide_gb300 as svw
    c = _case(3, [4, 1, 9], 2000, "bf16", nbias=0 if drop in ("bias", "all") else 6, masked=drop not in ("mask", "all"))
    over = {}
    if drop in ("history", "all"):
        c["history"], c["cu_h"], c["prompt"] = np.zeros(0, np.int32), np.zeros(4, np.int32), np.zeros(3, np.int32)
        over.update(history=None, cu_history=None, prompt_len=None)
    if drop in ("factors", "all"):
        c["rep"][:], c["freq"][:], c["pres"][:] = 1, 0, 0
        over.update(repetition=None, frequency=None, presence=None)
    a, kw = _args(c, **over)
    out = svw.logits_adjust(c["t"].cuda(), *a, **kw)
    _compare(out, c)
    if drop == "all":  # nothing to do: a copy, bit for bit
        import torch
        assert torch.equal(out.cpu().view(torch.int16), c["t"].view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [1000, 2003])
@pytest.mark.parametrize("pad_in,pad_out,off", [(8, 8, 0), (0, 24, 0), (5, 3, 0), (0, 0, 1), (1, 1, 3), (16, 16, 8)])
def test_adjust_strides_and_alignment(dtype, V, pad_in, pad_out, off):
    import serving_vocab_wide_gb300 as svw
    import torch
    c = _case(7, [3, 6], V, dtype)
    rows, t = c["rows"], c["t"]
    place = lambda pad, at: torch.full((rows * (V + pad) + at + 8,), 77.0, dtype=t.dtype, device="cuda")
    bi, bo = place(pad_in, off), place(pad_out, off)
    x = torch.as_strided(bi, (rows, V), (V + pad_in, 1), off)
    y = torch.as_strided(bo, (rows, V), (V + pad_out, 1), off)
    x.copy_(t)
    a, kw = _args(c)
    svw.logits_adjust(x, *a, out=y, **kw)
    _compare(y, c)
    y.fill_(77.0)
    assert bool((bo == 77.0).all()), "nothing outside the rows is written"
    assert torch.equal(x.cpu().view(torch.int16 if dtype == "bf16" else torch.int32),
                       t.view(torch.int16 if dtype == "bf16" else torch.int32))


def test_adjust_offsets_beyond_32_bits():
    import serving_vocab_wide_gb300 as svw
    import torch
    V, pitch = 1000, (1 << 28) + 8
    c = _case(9, [9], V, "bf16")  # the last row starts beyond 2^31 elements
    buf = torch.empty(9 * pitch + V, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (10, V), (pitch, 1))
    x.copy_(c["t"])
    a, kw = _args(c)
    _compare(svw.logits_adjust(x, *a, **kw), c)
    svw.logits_adjust(x, *a, out=x, **kw)
    _compare(x, c)


def test_adjust_nan_only_where_it_was():
    """NaN logits stay NaN where they are allowed, and vanish where the mask
    hides them; their neighbours are untouched."""
    import serving_vocab_wide_gb300 as svw
    c = _case(21, [5, 2], 3001, "bf16")
    c["t"][:, ::7] = float("nan")
    c["x"] = c["t"].double().numpy()
    a, kw = _args(c)
    _compare(svw.logits_adjust(c["t"].cuda(), *a, **kw), c)


def _bad(c, which, V):
    """Plants one bad value for request 1; the others stay good."""
    over = {}
    if which == "history token":
        c["history"][c["cu_h"][1]] = V
    elif which == "negative history token":
        c["history"][c["cu_h"][1]] = -1
    elif which == "draft token":
        c["tokens"][c["cu"][1]] = V + 3
    elif which == "prompt":
        c["prompt"][1] = c["cu_h"][2] - c["cu_h"][1] + 1
    elif which == "repetition":
        c["rep"][1] = 0
    elif which == "frequency":
        c["freq"][1] = np.nan
    elif which == "presence":
        c["pres"][1] = np.inf
    elif which == "bias token":
        c["biases"][1][0] = (V, 1.0)
    elif which == "bias value":
        c["biases"][1][0] = (0, np.inf)
    return over


@pytest.mark.parametrize("which", ["history token", "negative history token", "draft token", "prompt", "repetition",
                                   "frequency", "presence", "bias token", "bias value"])
def test_adjust_bad_request_becomes_nan(which):
    import serving_vocab_wide_gb300 as svw
    import torch
    V = 9000
    c = _case(31, [2, 3, 4], V, "bf16", hist=(5, 50))
    good = _reference(c)[0]
    _bad(c, which, V)
    a, kw = _args(c)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = svw.logits_adjust(c["t"].cuda(), *a, status=status, **kw).double().cpu().numpy()
    assert svw.device_status(int(status)) == svw.SVW_ERR_BAD_INPUT
    mine = slice(c["cu"][1] + 1, c["cu"][2] + 2)
    assert np.isnan(out[mine]).all()
    for s in (slice(0, c["cu"][1] + 1), slice(c["cu"][2] + 2, None)):
        assert np.array_equal(np.isnan(out[s]), np.isnan(good[s]))
        assert np.allclose(out[s], good[s], rtol=1e-2, atol=1e-2, equal_nan=True)


def test_adjust_bad_mask_row_and_offsets():
    import serving_vocab_wide_gb300 as svw
    import torch
    c = _case(33, [2, 3], 700, "fp32")
    for val in (4, -2):
        c["mask_row"][1] = val
        a, kw = _args(c)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = svw.logits_adjust(c["t"].cuda(), *a, status=status, **kw)
        assert int(status) == svw.SVW_DEV_BAD_INPUT
        assert bool(out[1].isnan().all()) and not bool(out[2].isnan().any())
    c["mask_row"][1] = 0
    a, kw = _args(c)
    cu = a[0].clone()
    cu[1] = -3  # both requests' ranges are wrong: nothing of them is written
    out = torch.full_like(c["t"].cuda(), 5.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    svw.logits_adjust(c["t"].cuda(), cu, a[1], out=out, status=status, **kw)
    assert int(status) == svw.SVW_DEV_BAD_INPUT and bool((out == 5.0).all())


def test_adjust_stream_and_graph():
    import serving_vocab_wide_gb300 as svw
    import torch
    c = _case(41, [4, 8], 12345, "bf16")
    a, kw = _args(c)
    x = c["t"].cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = svw.logits_adjust(x, *a, stream=s, **kw)
    s.synchronize()
    _compare(out, c)
    out.zero_()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        svw.logits_adjust(x, *a, out=out, **kw)
    g.replay()
    torch.cuda.synchronize()
    _compare(out, c)


def test_adjusted_logits_are_verified():
    """The masked and banned tokens are never emitted, and a position whose
    grammar allows one token emits it."""
    import serving_vocab_wide_gb300 as svw
    import torch
    c = _case(51, [4, 2, 7], 4000, "bf16", nbias=0)
    c["t"] = torch.randn(c["rows"], 4000).to(torch.bfloat16)
    c["mask"][:] = False
    only = [17, 1999, 3999]
    for k, v in enumerate(only):
        c["mask"][k, v] = True
    c["mask_row"] = np.repeat(np.arange(3), [5, 3, 8]).astype(np.int32)
    a, kw = _args(c)
    y = svw.logits_adjust(c["t"].cuda(), *a, **kw)
    R = int(c["cu"][-1])
    draft = torch.randn(R, 4000, device="cuda").to(torch.bfloat16)
    for T in (0.0, 1.0):
        acc, nxt = svw.spec_verify(y, draft, a[0], a[1], T, 3, total_draft_rows=R)
        tok = c["tokens"]
        for i in range(3):
            mine = tok[c["cu"][i]:c["cu"][i + 1]]
            want = 0
            while want < len(mine) and mine[want] == only[i]:
                want += 1
            assert int(nxt[i]) == only[i] and int(acc[i]) == want


def test_adjust_refusals():
    import serving_vocab_wide_gb300 as svw
    import torch
    c = _case(61, [4, 2], 640, "bf16")
    a, kw = _args(c)
    x = c["t"].cuda()
    E = svw.SvwError
    for wrong in ({"cu_history": None}, {"bias_values": None}, {"mask": None}, {"repetition": kw["repetition"][:1]},
                  {"repetition": kw["repetition"].double()}, {"history": kw["history"].long()},
                  {"mask": kw["mask"][:, :-1].contiguous()}, {"mask_row": kw["mask_row"][:-1]},
                  {"out": x[:, :-1]}, {"out": x.float()}, {"has_bonus": False}, {"mask_row": None},
                  {"history": kw["history"].cpu()}, {"total_draft_rows": 5}):
        with pytest.raises(E):
            svw.logits_adjust(x, *a, **{**kw, **wrong})
    with pytest.raises(E):
        svw.logits_adjust(x.half(), *a, **kw)
    with pytest.raises(E):
        svw.logits_adjust(x.t().contiguous().t(), *a, **kw)
    with pytest.raises(E):
        svw.logits_adjust(x.cpu(), *a, **kw)
    # an output that overlaps the input without being it
    big = torch.zeros(x.numel() + 64, dtype=x.dtype, device="cuda")
    with pytest.raises(E):
        svw.logits_adjust(big[:x.numel()].view(x.shape), *a, out=big[64:].view(x.shape), **kw)


@pytest.mark.parametrize("V,hist,lens", [(151936, 20000, [4]), (9000, 30000, [2, 3]), (4097, 5000, [1]),
                                         (151936, 7000, [1, 0, 2])])
def test_adjust_long_histories(V, hist, lens):
    """Histories of more distinct tokens than are counted at once."""
    import serving_vocab_wide_gb300 as svw
    assert svw.logits_adjust_workspace_size(len(lens), V, sum(lens), hist * len(lens), 0) > 0
    c = _case(71, lens, V, "bf16", hist=(hist, hist), nbias=300)
    rng = np.random.default_rng(72)
    c["history"] = rng.integers(0, V, len(c["history"])).astype(np.int32)
    a, kw = _args(c)
    import torch
    x = c["t"].cuda()
    out = svw.logits_adjust(x, *a, **kw)
    _compare(out, c)
    svw.logits_adjust(x, *a, out=x, **kw)
    assert torch.equal(out.view(torch.int16), x.view(torch.int16))


def test_adjust_bad_requests_of_a_large_batch():
    """The same refusals where the lists are counted first: a bad request's rows
    are NaN, a list that begins before an earlier one's end is bad, the others
    are right; a workspace of the caller's, whatever it holds."""
    import serving_vocab_wide_gb300 as svw
    import torch
    V, N = 5000, 600
    for which in ("history token", "draft token", "repetition", "bias value", "overlap"):
        c = _case(81, [1, 2] * (N // 2), V, "bf16", hist=(5, 30))
        good = _reference(c)
        bad = 1
        if which == "overlap":
            c["cu_h"][100] = c["cu_h"][98]  # request 99 runs backwards, request 100 begins inside an earlier one
            bad = None
        else:
            _bad(c, which, V)
        a, kw = _args(c)
        need = svw.logits_adjust_workspace_size(N, V, int(c["cu"][-1]), len(c["history"]), 5 * N)
        assert need > 0
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = svw.logits_adjust(c["t"].cuda(), *a, status=status, workspace=ws, **kw)
        assert int(status) == svw.SVW_DEV_BAD_INPUT
        mine = np.zeros(c["rows"], bool)  # the bad requests' rows
        for i in (99, 100) if bad is None else (bad,):
            mine[c["cu"][i] + i:c["cu"][i + 1] + i + 1] = True
        assert bool(out[torch.from_numpy(mine).cuda()].isnan().all()), which
        _compare(out, c, good, ~mine)
    with pytest.raises(svw.SvwError):
        svw.logits_adjust(c["t"].cuda(), *a, workspace=ws[:need - 1], **kw)


@pytest.mark.parametrize("requests", [2, 900])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_adjust_a_bias_of_zero_is_added(requests, dtype):
    """-0 with a bias of +0 is +0, in small batches, large ones and in place; with
    a bias of -0, or none, it stays -0."""
    import serving_vocab_wide_gb300 as svw
    import torch
    V, N = 8200, requests
    x = torch.full((N, V), -0.0, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    cu = i32([0] * (N + 1))
    kw = {"bias_tokens": i32([5, 4097, 8199] * N), "bias_values": torch.tensor([0.0, -0.0, 0.0] * N, device="cuda"),
          "cu_bias": i32([3 * n for n in range(N + 1)]), "total_draft_rows": 0}
    assert (svw.logits_adjust_workspace_size(N, V, 0, 0, 3 * N) > 0) == (N > 2)
    want = torch.zeros_like(x).copysign(x)
    want[:, [5, 8199]] = 0.0
    for out in (svw.logits_adjust(x, cu, **kw), svw.logits_adjust(x, cu, out=x, **kw)):
        assert bool((out == 0).all()) and torch.equal(torch.signbit(out), torch.signbit(want))


# ---------------------------------------------------------------------------
# batches whose lists are counted first
# ---------------------------------------------------------------------------
def _large(c):
    import serving_vocab_wide_gb300 as svw
    return svw.logits_adjust_workspace_size(len(c["cu"]) - 1, c["V"], int(c["cu"][-1]), len(c["history"]),
                                            sum(map(len, c["biases"]))) > 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [20000, 20003])
@pytest.mark.parametrize("pad_in,pad_out,off_in,off_out", [(8, 8, 0, 0), (5, 3, 0, 0), (16, 0, 1, 1), (1, 1, 3, 3), (8, 8, 0, 1)])
def test_adjust_large_strides_and_alignment(dtype, V, pad_in, pad_out, off_in, off_out):
    """Rows of any pitch and start, lying alike or differently, apart and in place."""
    import serving_vocab_wide_gb300 as svw
    import torch
    c = _case(13, [3, 2, 3] * 50, V, dtype, hist=(0, 60))
    assert _large(c)
    rows, t = c["rows"], c["t"]
    ints = torch.int16 if dtype == "bf16" else torch.int32
    place = lambda pad, at: torch.full((rows * (V + pad) + at + 8,), 77.0, dtype=t.dtype, device="cuda")
    bi, bo = place(pad_in, off_in), place(pad_out, off_out)
    x = torch.as_strided(bi, (rows, V), (V + pad_in, 1), off_in)
    y = torch.as_strided(bo, (rows, V), (V + pad_out, 1), off_out)
    x.copy_(t)
    a, kw = _args(c)
    svw.logits_adjust(x, *a, out=y, **kw)
    _compare(y, c)
    assert torch.equal(x.cpu().view(ints), t.view(ints))
    apart = y.clone()
    svw.logits_adjust(x, *a, out=x, **kw)
    assert torch.equal(x.contiguous().view(ints), apart.view(ints))
    for buf, v in ((bo, y), (bi, x)):
        v.fill_(77.0)
        assert bool((buf == 77.0).all()), "nothing outside the rows is written"


@pytest.mark.parametrize("dtype,lens,V", [("bf16", [2, 0, 5], 262208), ("fp32", [3, 1], 262209), ("bf16", [4] * 9, 1 << 20)])
def test_adjust_vocabularies_of_several_ranges(dtype, lens, V):
    """The lists' bitmap holds 2^18 tokens at a time."""
    import serving_vocab_wide_gb300 as svw
    import torch
    c = _case(91, lens, V, dtype, hist=(5000, 9000), nbias=40)
    rng = np.random.default_rng(92)
    h = rng.integers(0, V, len(c["history"])).astype(np.int32)
    h[::97] = rng.integers(max(0, V - 200), V, len(h[::97]))  # the last range, and both sides of a boundary
    h[1::89] = (1 << 18) + rng.integers(-3, 3, len(h[1::89]))
    c["history"] = h
    c["tokens"][0] = 1 << 18
    assert _large(c)
    a, kw = _args(c)
    x = c["t"].cuda()
    out = svw.logits_adjust(x, *a, **kw)
    _compare(out, c)
    svw.logits_adjust(x, *a, out=x, **kw)
    ints = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(out.view(ints), x.view(ints))


@pytest.mark.parametrize("in_place", [False, True])
def test_adjust_large_graph_and_streams(in_place):
    """The two launches captured and replayed with other logits and histories,
    and on two streams at once."""
    import serving_vocab_wide_gb300 as svw
    import torch
    c = _case(43, [3, 5, 0] * 60, 15001, "bf16", hist=(0, 90))
    assert _large(c)
    a, kw = _args(c)
    x = c["t"].cuda()
    want = svw.logits_adjust(x, *a, **kw)
    buf = x.clone()
    out = buf if in_place else torch.zeros_like(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svw.logits_adjust(buf, *a, out=out, **kw)
    other = x.flip(1).contiguous()
    history = kw["history"].clone()
    for n in range(4):
        src = x if n % 2 == 0 else other
        kw["history"].copy_(history if n < 2 else history.flip(0))
        buf.copy_(src)
        g.replay()
        fresh = svw.logits_adjust(src, *a, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), fresh.view(torch.int16)), n
    kw["history"].copy_(history)
    copies = [x.clone() for _ in range(4)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()] * 2
    torch.cuda.synchronize()
    got = [svw.logits_adjust(y, *a, stream=s, out=y if in_place else None, **kw) for y, s in zip(copies, streams)]
    torch.cuda.synchronize()
    for y in got:
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("in_place", [False, True])
def test_adjust_large_bad_mask_rows_and_nan(in_place):
    """Mask rows out of range make their rows NaN, and only those; NaN logits
    vanish where a mask hides them."""
    import serving_vocab_wide_gb300 as svw
    import torch
    c = _case(35, [2, 3, 1] * 120, 12001, "bf16", hist=(0, 50))
    assert _large(c)
    c["t"][:, ::7] = float("nan")
    c["x"] = c["t"].double().numpy()
    good = _reference(c)
    bad = np.zeros(c["rows"], bool)
    for r, v in ((5, 4), (77, -2), (c["rows"] - 1, 1 << 30)):
        c["mask_row"][r], bad[r] = v, True
    a, kw = _args(c)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = c["t"].cuda()
    out = svw.logits_adjust(x, *a, status=status, out=x if in_place else None, **kw)
    assert int(status) == svw.SVW_DEV_BAD_INPUT
    assert bool(out[torch.from_numpy(bad).cuda()].isnan().all())
    _compare(out, c, good, ~bad)


def test_adjust_large_offsets_beyond_32_bits():
    import serving_vocab_wide_gb300 as svw
    import torch
    V, pitch = 60000, (1 << 24) + 8
    c = _case(9, [9] * 18, V, "bf16", hist=(0, 100))  # the last rows start beyond 2^31 elements
    assert _large(c) and (c["rows"] - 1) * pitch > 1 << 31
    buf = torch.empty((c["rows"] - 1) * pitch + V, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (c["rows"], V), (pitch, 1))
    x.copy_(c["t"])
    a, kw = _args(c)
    want = _reference(c)
    _compare(svw.logits_adjust(x, *a, **kw), c, want)
    svw.logits_adjust(x, *a, out=x, **kw)
    _compare(x, c, want)
