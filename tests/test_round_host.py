"""What the Python calls of a verification round do on the host, with stand-ins
for the GPU's tensors and streams: where memory is taken, on which device they
launch, what they hand to the library."""
import contextlib
import ctypes
import types

import pytest
import torch

import serving_vocab_wide_gb300 as svw

I32, F32, BF16, U8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8


class Tensor:
    """A tensor's shape and place, nothing in it."""

    def __init__(self, shape, dtype, pool="program", gpu=0):
        self.shape, self.dtype, self.pool, self.gpu, self.recorded = tuple(shape), dtype, pool, gpu, []
        self.device = f"cuda:{gpu}"

    def stride(self, d=None):
        s = [1] * len(self.shape)
        for i in range(len(s) - 2, -1, -1):
            s[i] = s[i + 1] * self.shape[i + 1]
        return tuple(s) if d is None else s[d]

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.gpu

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def record_stream(self, s):
        self.recorded.append(s)


class Stream:
    def __init__(self, handle, gpu=0):
        self.cuda_stream, self.device_index, self.device = handle, gpu, torch.device("cuda", gpu)


@pytest.fixture
def host(monkeypatch):
    """The calls recorded; new tensors know the stream whose pool they came from."""
    svw.build()
    real = svw.lib()
    h = types.SimpleNamespace(current=Stream(7), device=0, made=[], calls=[])

    @contextlib.contextmanager
    def stream(s):
        before, h.current = h.current, s
        yield
        h.current = before

    def empty(shape, dtype, device):
        t = Tensor((shape,) if isinstance(shape, int) else shape, dtype, h.current)
        h.made.append(t)
        return t

    class Lib:
        def __getattr__(self, name):
            if name in ("logits_adjust", "kv_append", "paged_attention"):
                return lambda *a: h.calls.append((name, a)) or 0
            return getattr(real, name)

    cuda = types.SimpleNamespace(stream=stream, current_stream=lambda device=None: h.current,
                                 current_device=lambda: h.device)
    c = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda gpu: h.current.cuda_stream,
                              _cuda_getDevice=lambda: h.device)
    fake = types.SimpleNamespace(int32=I32, float32=F32, uint8=U8, bfloat16=BF16, empty=empty, cuda=cuda, _C=c)
    monkeypatch.setattr(svw, "_torch", lambda: fake)
    monkeypatch.setattr(svw, "lib", lambda: Lib())
    return h


def _calls(gpu=0, **kw):
    """Each operator on a batch whose outputs and workspaces it makes itself."""
    t = lambda shape, dtype: Tensor(shape, dtype, gpu=gpu)
    where = (t((10, 2, 16, 64), BF16), t((10, 2, 16, 64), BF16), t((3, 4), I32), t((4,), I32), t((3,), I32))
    q, k, v = t((9, 4, 64), BF16), t((9, 2, 64), BF16), t((9, 2, 64), BF16)
    big = 500
    x = t((4 * big, 65536), BF16)
    return {
        "paged_attention": lambda: svw.paged_attention(q, *where, **kw),
        "kv_append": lambda: svw.kv_append(k, v, *where, q=q, **kw),
        "logits_adjust": lambda: svw.logits_adjust(x, t((big + 1,), I32), t((3 * big,), I32),
                                                   total_draft_rows=3 * big, **kw),
    }


@pytest.mark.parametrize("name,outputs,workspaces", [("paged_attention", 2, 1), ("kv_append", 1, 0), ("logits_adjust", 1, 1)])
def test_memory_comes_from_the_stream_that_uses_it(host, name, outputs, workspaces):
    """Memory that the current stream gave back may still be in use on it: what
    another stream is to write comes from that stream's pool.  The outputs, which
    the program reads where it goes on, are the current stream's too."""
    side, current = Stream(9), host.current
    _calls(stream=side)[name]()
    assert len(host.made) == outputs + workspaces and host.current is current
    assert all(t.pool is side for t in host.made)
    assert host.calls[0][0] == name and host.calls[0][1][-1] == side.cuda_stream
    assert [t.dtype for t in host.made].count(U8) == workspaces
    for t in host.made:
        assert t.recorded == ([] if t.dtype is U8 else [current])
    # without a stream: the current one's, and nothing to record
    host.made.clear()
    _calls()[name]()
    assert all(t.pool is current and not t.recorded for t in host.made)
    assert host.calls[1][1][-1] == current.cuda_stream


@pytest.mark.parametrize("name", ["paged_attention", "kv_append", "logits_adjust"])
def test_another_gpu_than_the_current_one_is_refused(host, name):
    """The library launches on the current device: tensors or a stream of another
    one are refused before anything is taken or launched."""
    host.device = 1
    with pytest.raises(svw.SvwError, match="current"):
        _calls()[name]()
    host.device = 0
    with pytest.raises(svw.SvwError, match="current"):
        _calls(stream=Stream(9, gpu=1))[name]()
    assert not host.made and not host.calls
    _calls(stream=Stream(9))[name]()
    host.device = 1
    _calls(gpu=1, stream=Stream(11, gpu=1))[name]()
    assert len(host.calls) == 2


def test_the_cache_is_handed_over_whole():
    """The bytes of svw_paged_kv: as many as the library copies, each field in its place."""
    k, v, table = Tensor((10, 2, 16, 64), BF16), Tensor((10, 2, 16, 64), BF16), Tensor((3, 4), I32)
    k.data_ptr, v.data_ptr, table.data_ptr = (lambda: 0x1000), (lambda: 0x2000), (lambda: 0x3000)
    packed, gpu, shape = svw._paged(k, v, table, 3)
    assert len(packed) == ctypes.sizeof(svw._PagedKV) == 104
    c = svw._PagedKV.from_buffer_copy(packed)
    assert (c.k, c.v, c.block_table) == (0x1000, 0x2000, 0x3000)
    assert list(c.k_stride) == list(c.v_stride) == [2048, 1024, 64]
    assert (c.table_stride, c.max_pages, c.n_pages, c.page_size, c.n_kv_heads, c.head_dim) == (4, 4, 10, 16, 2, 64)
    assert gpu == 0 and shape == k.shape
