"""serving_vocab_wide_gb300 -- batched speculative verification and the OPD
loss over full-vocabulary logits, as hand-written CUDA for GB300 (sm_103a).

This module is a thin ctypes binding over the C ABI in ``include/svw.h``:
it only marshals PyTorch CUDA tensors (data pointers, sizes, the current
stream) into the library's entry points.  Every step of the computation runs
in the library's kernels; there is no CPU or PyTorch fallback -- if the shared
library is missing the calls raise.

Build the library with ``serving_vocab_wide_gb300.build()`` (nvcc, sm_103a).
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading

from .build import LIB_PATH, build  # noqa: F401

SVW_F32 = 0
SVW_BF16 = 1
SVW_DEV_BAD_INPUT = 1
SVW_DEV_TIMEOUT = 2
SVW_ERR_BAD_INPUT = 6
SVW_ERR_TIMEOUT = 7
SVW_MAX_LEN = 32

_lib = None
_lock = threading.Lock()


class SvwError(RuntimeError):
    pass


class _PagedKV(ctypes.Structure):
    """svw_paged_kv"""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_stride", ctypes.c_int64 * 3),
                ("v_stride", ctypes.c_int64 * 3), ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("max_pages", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


def lib():
    """The loaded shared library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise SvwError(f"CUDA library not built: {LIB_PATH} is missing "
                               "(run serving_vocab_wide_gb300.build())")
            L = ctypes.CDLL(LIB_PATH)
            P, I32, I64, F, U64, SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                       ctypes.c_float, ctypes.c_uint64, ctypes.c_size_t)
            L.svw_verify_workspace_size.argtypes = [I32, I64, I32, ctypes.c_int]
            L.svw_verify_workspace_size.restype = SZ
            L.svw_workspace_size.argtypes = [I32, I64, I32, I32]
            L.svw_workspace_size.restype = SZ
            L.svw_device_status.argtypes = [I32]
            L.svw_device_status.restype = ctypes.c_int
            L.spec_verify.argtypes = [P, P, ctypes.c_int, I32, I32, P, I64, I32, P, F, U64,
                                      P, P, P, P, SZ, P]
            L.spec_verify.restype = ctypes.c_int
            L.svw_verify_early_workspace_size.argtypes = [I32, I64, I32, ctypes.c_int]
            L.svw_verify_early_workspace_size.restype = SZ
            L.spec_verify_early.argtypes = [P, P, ctypes.c_int, I32, I32, P, I64, I32, P, F, U64,
                                            P, P, P, P, P, SZ, P]
            L.spec_verify_early.restype = ctypes.c_int
            L.svw_verify_filtered_workspace_size.argtypes = [I32, I64, I32, ctypes.c_int]
            L.svw_verify_filtered_workspace_size.restype = SZ
            L.spec_verify_filtered.argtypes = [P, P, ctypes.c_int, I32, I32, P, I64, I32, P, F, I32, F, U64,
                                               P, P, P, P, SZ, P]
            L.spec_verify_filtered.restype = ctypes.c_int
            L.svw_opd_workspace_size.argtypes = [I64]
            L.svw_opd_workspace_size.restype = SZ
            L.opd_loss.argtypes = [P, P, ctypes.c_int, I32, I32, P, I64, I32, F, F, F, F,
                                   P, P, P, P, SZ, P]
            L.opd_loss.restype = ctypes.c_int
            L.spec_verify_noalloc.argtypes = [P, P, ctypes.c_int, I32, I32, P, I64, I32, P, F, U64,
                                              P, P, P, P]
            L.svw_verify_opd_workspace_size.argtypes = [I32, I64, I32, ctypes.c_int]
            L.svw_verify_opd_workspace_size.restype = SZ
            L.spec_verify_opd.argtypes = [P, P, ctypes.c_int, I32, I32, P, I64, I32, P, F, F, U64, F, F, F,
                                          P, P, P, P, P, P, SZ, P]
            L.spec_verify_opd.restype = ctypes.c_int
            L.spec_verify_noalloc.restype = ctypes.c_int
            L.svw_length_head_workspace_size.argtypes = [I32, I32, I32]
            L.svw_length_head_workspace_size.restype = SZ
            L.length_head.argtypes = [P, P, P, P, F, I32, I32, I32, I32, F, P, P, P, SZ, P]
            L.length_head.restype = ctypes.c_int
            L.length_head_label.argtypes = [P, P, P, I32, P, P, P]
            L.length_head_label.restype = ctypes.c_int
            L.svw_logits_adjust_workspace_size.argtypes = [I32, I32, I64, I64, I64]
            L.svw_logits_adjust_workspace_size.restype = SZ
            L.logits_adjust.argtypes = [P, I64, ctypes.c_int, I32, I32, P, I64, I32, P, P, P, I64, P, P, P, P,
                                        P, P, P, I64, P, I64, P, P, I64, P, P, SZ, P]
            L.logits_adjust.restype = ctypes.c_int
            L.kv_append.argtypes = [P, I64, I64, P, I64, I64, P, I64, I64, P, ctypes.c_int, I32, I32, P, I64, P,
                                    P, P, I64, I32, I32, P, P, P]
            L.kv_append.restype = ctypes.c_int
            L.svw_paged_attention_workspace_size.argtypes = [I64, I32, I32, I32]
            L.svw_paged_attention_workspace_size.restype = SZ
            L.paged_attention.argtypes = [P, I64, I64, ctypes.c_int, I32, I32, P, I64, P, P, F, I32, I32, P, P, P,
                                          P, SZ, P]
            L.paged_attention.restype = ctypes.c_int
            L.svw_time_next_launch.argtypes = [ctypes.c_char_p, P, P]
            L.svw_time_next_launch.restype = ctypes.c_int
            L.svw_set_wait_limit.argtypes = [I64]
            L.svw_set_wait_limit.restype = ctypes.c_int
            L.svw_set_fault.argtypes = [I32]
            L.svw_set_fault.restype = ctypes.c_int
            L.svw_status_string.argtypes = [ctypes.c_int]
            L.svw_status_string.restype = ctypes.c_char_p
            L.svw_version.argtypes = []
            L.svw_version.restype = I32
            _lib = L
    return _lib


def _check(rc: int):
    if rc != 0:
        raise SvwError(lib().svw_status_string(rc).decode())


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return SVW_BF16
    if t.dtype == torch.float32:
        return SVW_F32
    raise SvwError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _stream_ptr(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise SvwError("tensors must be contiguous CUDA tensors")


def time_next_launch(kernel: str | None, begin=None, end=None):
    """Arm the library's one-shot timer: the next launch of `kernel` from this
    thread records the torch.cuda.Event `begin` before it and `end` after it
    on the launch stream (measurement only)."""
    if kernel is None:
        _check(lib().svw_time_next_launch(None, None, None))
        return
    for ev in (begin, end):
        if not ev.cuda_event:  # torch creates the CUDA event at its first record
            ev.record()
    _check(lib().svw_time_next_launch(kernel.encode(), ctypes.c_void_p(begin.cuda_event),
                                      ctypes.c_void_p(end.cuda_event)))


DEFAULT_WAIT_CYCLES = 4_000_000_000


def set_wait_limit(cycles: int = DEFAULT_WAIT_CYCLES):
    """Test hook: the deadline (SM cycles) of every bounded wait in the
    library's kernels on the current device."""
    _check(lib().svw_set_wait_limit(int(cycles)))


def set_fault(kind: int = 0):
    """Test hook: 1 = the next calls' stats / OPD fast kernels leave one CTA
    (cluster) without its copies, so that its first wait runs out; 0 = none."""
    _check(lib().svw_set_fault(int(kind)))


def workspace_size(n_requests: int, total_draft_rows: int, V: int, max_len: int = SVW_MAX_LEN) -> int:
    """One workspace size that serves every entry point on this batch shape."""
    return int(lib().svw_workspace_size(n_requests, total_draft_rows, V, max_len))


def device_status(word: int) -> int:
    """svw_status code of a device status word (SVW_ERR_TIMEOUT, SVW_ERR_BAD_INPUT or 0)."""
    return int(lib().svw_device_status(int(word)))


def verify_workspace_size(n_requests: int, total_draft_rows: int, V: int, dtype_code: int) -> int:
    return int(lib().svw_verify_workspace_size(n_requests, total_draft_rows, V, dtype_code))


def opd_workspace_size(total_draft_rows: int) -> int:
    return int(lib().svw_opd_workspace_size(total_draft_rows))


def spec_verify(target, draft, cu_draft, draft_tokens, temperature: float, seed: int,
                max_len: int = SVW_MAX_LEN, total_draft_rows: int | None = None,
                accept_len=None, next_token=None, status=None, workspace=None, stream=None):
    """Verify a ragged batch.  Returns (accept_len, next_token) int32 CUDA tensors.

    target: [total_draft_rows + N, V], draft: [total_draft_rows, V] (bf16 or
    fp32); cu_draft: int32 [N + 1] CSR offsets; draft_tokens: int32
    [total_draft_rows].  Output / workspace / status tensors may be passed in
    to avoid allocation; `total_draft_rows` (= cu_draft[-1]) may be passed to
    avoid a device read.
    """
    import torch
    _need_cuda(target, draft, cu_draft, draft_tokens)
    N = cu_draft.numel() - 1
    V = target.shape[-1]
    R = int(cu_draft[-1].item()) if total_draft_rows is None else int(total_draft_rows)
    code = _dtype_code(target)
    dev = target.device
    if accept_len is None:
        accept_len = torch.empty(N, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(N, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(1, verify_workspace_size(N, R, V, code)), dtype=torch.uint8,
                                device=dev)
    _need_cuda(accept_len, next_token, workspace, status)
    rc = lib().spec_verify(_ptr(target), _ptr(draft), code, V, N, _ptr(cu_draft), R, max_len,
                           _ptr(draft_tokens), float(temperature), int(seed) & (2**64 - 1),
                           _ptr(accept_len), _ptr(next_token), _ptr(status), _ptr(workspace),
                           workspace.numel(), _stream_ptr(stream))
    _check(rc)
    return accept_len, next_token


def verify_early_workspace_size(n_requests: int, total_draft_rows: int, V: int, dtype_code: int) -> int:
    return int(lib().svw_verify_early_workspace_size(n_requests, total_draft_rows, V, dtype_code))


def spec_verify_early(target, draft, cu_draft, draft_tokens, temperature: float, seed: int,
                      max_len: int = SVW_MAX_LEN, total_draft_rows: int | None = None,
                      accept_len=None, next_token=None, status=None, bytes_read=None, workspace=None,
                      stream=None):
    """spec_verify that stops reading each request at its first rejection.
    Same (accept_len, next_token); `bytes_read` (int64 CUDA scalar, optional)
    receives the logit bytes the call streamed."""
    import torch
    _need_cuda(target, draft, cu_draft, draft_tokens)
    N = cu_draft.numel() - 1
    V = target.shape[-1]
    R = int(cu_draft[-1].item()) if total_draft_rows is None else int(total_draft_rows)
    code = _dtype_code(target)
    dev = target.device
    if accept_len is None:
        accept_len = torch.empty(N, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(N, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(1, verify_early_workspace_size(N, R, V, code)), dtype=torch.uint8,
                                device=dev)
    _need_cuda(accept_len, next_token, workspace, status, bytes_read)
    if bytes_read is not None and (bytes_read.dtype != torch.int64 or bytes_read.numel() != 1):
        raise SvwError("bytes_read must be a one-element int64 tensor")
    rc = lib().spec_verify_early(_ptr(target), _ptr(draft), code, V, N, _ptr(cu_draft), R, max_len,
                                 _ptr(draft_tokens), float(temperature), int(seed) & (2**64 - 1),
                                 _ptr(accept_len), _ptr(next_token), _ptr(status), _ptr(bytes_read),
                                 _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    _check(rc)
    return accept_len, next_token


SVW_FILTER_MAX_K = 1024


def verify_filtered_workspace_size(n_requests: int, total_draft_rows: int, V: int, dtype_code: int) -> int:
    return int(lib().svw_verify_filtered_workspace_size(n_requests, total_draft_rows, V, dtype_code))


def spec_verify_filtered(target, draft, cu_draft, draft_tokens, temperature: float, top_k: int, top_p: float,
                         seed: int, max_len: int = SVW_MAX_LEN, total_draft_rows: int | None = None,
                         accept_len=None, next_token=None, status=None, workspace=None, stream=None):
    """spec_verify with both distributions top-k / top-p filtered (draft tokens
    drawn from the filtered draft distribution).  Returns (accept_len, next_token)."""
    import torch
    _need_cuda(target, draft, cu_draft, draft_tokens)
    N = cu_draft.numel() - 1
    V = target.shape[-1]
    R = int(cu_draft[-1].item()) if total_draft_rows is None else int(total_draft_rows)
    code = _dtype_code(target)
    dev = target.device
    if accept_len is None:
        accept_len = torch.empty(N, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(N, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(1, verify_filtered_workspace_size(N, R, V, code)), dtype=torch.uint8,
                                device=dev)
    _need_cuda(accept_len, next_token, workspace, status)
    rc = lib().spec_verify_filtered(_ptr(target), _ptr(draft), code, V, N, _ptr(cu_draft), R, max_len,
                                    _ptr(draft_tokens), float(temperature), int(top_k), float(top_p),
                                    int(seed) & (2**64 - 1), _ptr(accept_len), _ptr(next_token), _ptr(status),
                                    _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    _check(rc)
    return accept_len, next_token


def spec_verify_noalloc(target, draft, cu_draft, draft_tokens, temperature: float, seed: int,
                        max_len: int = SVW_MAX_LEN, total_draft_rows: int | None = None,
                        accept_len=None, next_token=None, status=None, stream=None):
    """spec_verify on the library's fixed per-GPU scratch instead of a caller
    workspace (for callers that cannot allocate).  Calls that may overlap on
    the GPU share that scratch and must be serialised on one stream."""
    import torch
    _need_cuda(target, draft, cu_draft, draft_tokens)
    N = cu_draft.numel() - 1
    V = target.shape[-1]
    R = int(cu_draft[-1].item()) if total_draft_rows is None else int(total_draft_rows)
    dev = target.device
    if accept_len is None:
        accept_len = torch.empty(N, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(N, dtype=torch.int32, device=dev)
    _need_cuda(accept_len, next_token, status)
    # the library uses the current device's scratch: make the inputs' device current
    with torch.cuda.device(dev):
        rc = lib().spec_verify_noalloc(_ptr(target), _ptr(draft), _dtype_code(target), V, N,
                                       _ptr(cu_draft), R, max_len, _ptr(draft_tokens),
                                       float(temperature), int(seed) & (2**64 - 1), _ptr(accept_len),
                                       _ptr(next_token), _ptr(status), _stream_ptr(stream))
    _check(rc)
    return accept_len, next_token


def verify_opd_workspace_size(n_requests: int, total_draft_rows: int, V: int, dtype_code: int) -> int:
    return int(lib().svw_verify_opd_workspace_size(n_requests, total_draft_rows, V, dtype_code))


def spec_verify_opd(target, draft, cu_draft, draft_tokens, temperature: float, seed: int,
                    opd_temperature: float | None = None, clip_c: float = 1.0, lambda_ce: float = 0.1,
                    grad_scale: float = 1.0, max_len: int = SVW_MAX_LEN,
                    total_draft_rows: int | None = None, want_grad: bool = True, accept_len=None,
                    next_token=None, loss=None, dlogits=None, status=None, workspace=None, stream=None):
    """Verification and the OPD loss on the same batch in one pass.  Returns
    (accept_len, next_token, loss, dlogits or None).  opd_temperature
    defaults to temperature (or 1.0 when greedy)."""
    import torch
    _need_cuda(target, draft, cu_draft, draft_tokens)
    N = cu_draft.numel() - 1
    V = target.shape[-1]
    R = int(cu_draft[-1].item()) if total_draft_rows is None else int(total_draft_rows)
    code = _dtype_code(target)
    dev = target.device
    if opd_temperature is None:
        opd_temperature = temperature if temperature > 0 else 1.0
    if accept_len is None:
        accept_len = torch.empty(N, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(N, dtype=torch.int32, device=dev)
    if loss is None:
        loss = torch.empty(R, dtype=torch.float32, device=dev)
    if want_grad and dlogits is None:
        dlogits = torch.empty((R, V), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(1, verify_opd_workspace_size(N, R, V, code)), dtype=torch.uint8,
                                device=dev)
    _need_cuda(accept_len, next_token, loss, dlogits, status, workspace)
    rc = lib().spec_verify_opd(_ptr(target), _ptr(draft), code, V, N, _ptr(cu_draft), R, max_len,
                               _ptr(draft_tokens), float(temperature), float(opd_temperature),
                               int(seed) & (2**64 - 1), float(clip_c), float(lambda_ce),
                               float(grad_scale), _ptr(accept_len), _ptr(next_token), _ptr(loss),
                               _ptr(dlogits) if want_grad else None, _ptr(status), _ptr(workspace),
                               workspace.numel(), _stream_ptr(stream))
    _check(rc)
    return accept_len, next_token, loss, (dlogits if want_grad else None)


def length_head(hidden, w1, b1, w2, b2: float, gamma: float = 1.0, a_hat=None, k_hat=None, workspace=None,
                stream=None):
    """Adaptive length head forward.  hidden: bf16 [N, k, H], w1: bf16 [H', H],
    b1, w2: float32 [H'].  Returns (a_hat float32 [N], k_hat int32 [N])."""
    import torch
    _need_cuda(hidden, w1, b1, w2)
    if hidden.dtype != torch.bfloat16 or w1.dtype != torch.bfloat16:
        raise SvwError("hidden states and W1 must be bfloat16")
    N, k, H = hidden.shape
    Hp = w1.shape[0]
    dev = hidden.device
    if a_hat is None:
        a_hat = torch.empty(N, dtype=torch.float32, device=dev)
    if k_hat is None:
        k_hat = torch.empty(N, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(1, int(lib().svw_length_head_workspace_size(N, k, Hp))), dtype=torch.uint8,
                                device=dev)
    _need_cuda(a_hat, k_hat, workspace)
    rc = lib().length_head(_ptr(hidden), _ptr(w1), _ptr(b1), _ptr(w2), float(b2), N, k, H, Hp, float(gamma),
                           _ptr(a_hat), _ptr(k_hat), _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    _check(rc)
    return a_hat, k_hat


def length_head_label(accept_len, cu_draft, a_hat=None, a_star=None, loss=None, stream=None):
    """a* = accept_len / L per request and, with a_hat, the MSE (a_hat - a*)^2."""
    import torch
    _need_cuda(accept_len, cu_draft, a_hat)
    N = accept_len.numel()
    dev = accept_len.device
    if a_star is None:
        a_star = torch.empty(N, dtype=torch.float32, device=dev)
    if a_hat is not None and loss is None:
        loss = torch.empty(N, dtype=torch.float32, device=dev)
    _need_cuda(a_star, loss)
    rc = lib().length_head_label(_ptr(accept_len), _ptr(cu_draft), _ptr(a_hat), N, _ptr(a_star), _ptr(loss),
                                 _stream_ptr(stream))
    _check(rc)
    return a_star, loss


def opd_loss(target, draft, temperature: float = 1.0, clip_c: float = 1.0,
             lambda_ce: float = 0.1, grad_scale: float = 1.0, cu_draft=None,
             has_bonus: bool = False, want_grad: bool = True, loss=None, dlogits=None,
             status=None, workspace=None, exact_only: bool = False, stream=None):
    """Clipped reverse-KL + lambda*CE per draft row, and its gradient wrt the
    draft logits.  Returns (loss [R] fp32, dlogits [R, V] fp32 or None).

    A workspace (uint8, >= opd_workspace_size(R) bytes) is allocated when not
    given; exact_only=True passes none, so that every row takes the exact
    three-pass kernel."""
    import torch
    _need_cuda(target, draft, cu_draft)
    R, V = draft.shape
    code = _dtype_code(draft)
    N = (cu_draft.numel() - 1) if has_bonus else 0
    dev = draft.device
    if loss is None:
        loss = torch.empty(R, dtype=torch.float32, device=dev)
    if want_grad and dlogits is None:
        dlogits = torch.empty((R, V), dtype=torch.float32, device=dev)
    if exact_only:
        workspace = None
    elif workspace is None:
        workspace = torch.empty(max(1, opd_workspace_size(R)), dtype=torch.uint8, device=dev)
    _need_cuda(loss, dlogits, status, workspace)
    rc = lib().opd_loss(_ptr(target), _ptr(draft), code, V, N, _ptr(cu_draft) if has_bonus else None,
                        R, 1 if has_bonus else 0, float(temperature), float(clip_c),
                        float(lambda_ce), float(grad_scale), _ptr(loss),
                        _ptr(dlogits) if want_grad else None, _ptr(status), _ptr(workspace),
                        0 if workspace is None else workspace.numel(), _stream_ptr(stream))
    _check(rc)
    return loss, (dlogits if want_grad else None)


def _need_like(index, dtype, names, ts):
    """Each given tensor is contiguous, of this type and on this GPU."""
    for name, t in zip(names, ts):
        if t is not None and (t.dtype != dtype or t.get_device() != index or not t.is_contiguous()):
            raise SvwError(f"{name} must be a contiguous {dtype} tensor on cuda:{index}")


def _off(t, dtype, index):
    """Whether a tensor is not contiguous, of this type and on this GPU (None is fine)."""
    return t is not None and (t.dtype is not dtype or t.get_device() != index or not t.is_contiguous())


def _addr(t):
    return 0 if t is None else t.data_ptr()


def _stream_of(stream, index):
    """The handle of `stream`, or of the current stream of GPU `index`."""
    return _torch()._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


@functools.lru_cache(maxsize=None)
def _torch():
    import torch
    return torch


def _need_current(stream, gpu):
    """The library launches on the current device: the tensors' GPU has to be it, and the stream's."""
    if _torch()._C._cuda_getDevice() != gpu or (stream is not None and stream.device.index != gpu):
        raise SvwError(f"cuda:{gpu} must be the current device, and the stream's")


def _empty(stream, gpu, shape, dtype, device, returned=True):
    """An empty tensor to be written on `stream` (None: the current one).  It
    comes from that stream's pool: what the current stream has given back may
    still be in use there.  The program reads what is returned to it on the
    current stream, so it is reused only after that one is done with it too."""
    torch = _torch()
    if stream is None or stream.cuda_stream == torch._C._cuda_getCurrentRawStream(gpu):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


@functools.lru_cache(maxsize=64)
def logits_adjust_workspace_size(n_requests: int, V: int, total_draft_rows: int, total_history: int,
                                 total_bias: int) -> int:
    return int(lib().svw_logits_adjust_workspace_size(n_requests, V, total_draft_rows, total_history, total_bias))


def logits_adjust(logits, cu_draft, draft_tokens=None, *, history=None, cu_history=None, prompt_len=None,
                  repetition=None, frequency=None, presence=None, bias_tokens=None, bias_values=None, cu_bias=None,
                  mask=None, mask_row=None, has_bonus: bool = True, total_draft_rows: int | None = None, out=None,
                  status=None, workspace=None, stream=None):
    """Penalties for repeated tokens, biases and grammar masks on the logits of
    every drafted position (a position has seen the request's history and the
    drafted tokens before it).  Returns the adjusted logits.

    logits: [total_draft_rows + N, V] (the verify layout; [total_draft_rows, V]
    with has_bonus=False), bf16 or fp32, rows any pitch apart; cu_draft, the
    other cu_*: int32 CSR offsets; history, prompt_len, bias_tokens, mask_row:
    int32; repetition, frequency, presence, bias_values: float32; mask: int32
    [mask rows, ceil(V / 32)] of 32 tokens' bits each, the row of each logit row
    in mask_row (-1: unmasked; without mask_row, its own).  out may be logits
    (in place).  `total_draft_rows` (= cu_draft[-1]) may be passed to avoid a
    device read; workspace: uint8, >= logits_adjust_workspace_size(...) bytes.
    """
    torch = _torch()
    i32, f32 = torch.int32, torch.float32
    code = _dtype_code(logits)
    gpu = logits.get_device()
    if gpu < 0 or logits.dim() != 2 or logits.stride(1) != 1:
        raise SvwError("logits must be a CUDA matrix with contiguous rows")
    _need_current(stream, gpu)
    rows, V = logits.shape
    N = cu_draft.numel() - 1
    R = int(cu_draft[-1].item()) if total_draft_rows is None else int(total_draft_rows)
    if rows != R + (N if has_bonus else 0):
        raise SvwError(f"logits have {rows} rows for {R} draft rows of {N} requests")
    if (_off(cu_draft, i32, gpu) or _off(draft_tokens, i32, gpu) or _off(repetition, f32, gpu)
            or _off(frequency, f32, gpu) or _off(presence, f32, gpu) or _off(status, i32, gpu)):
        _need_like(gpu, i32, ("cu_draft", "draft_tokens", "status"), (cu_draft, draft_tokens, status))
        _need_like(gpu, f32, ("repetition", "frequency", "presence"), (repetition, frequency, presence))
    if ((repetition is not None and repetition.numel() != N) or (frequency is not None and frequency.numel() != N)
            or (presence is not None and presence.numel() != N)):
        raise SvwError(f"repetition, frequency and presence must have {N} elements")
    if draft_tokens is not None and draft_tokens.numel() != R:
        raise SvwError(f"draft_tokens must have {R} elements")
    if (history is None) is not (cu_history is None) or (prompt_len is not None and history is None):
        raise SvwError("history comes with cu_history, prompt_len with a history")
    n_history = n_bias = mask_rows = 0
    if history is not None:
        if _off(history, i32, gpu) or _off(cu_history, i32, gpu) or _off(prompt_len, i32, gpu):
            _need_like(gpu, i32, ("history", "cu_history", "prompt_len"), (history, cu_history, prompt_len))
        if cu_history.numel() != N + 1 or (prompt_len is not None and prompt_len.numel() != N):
            raise SvwError(f"cu_history must have {N + 1} elements, prompt_len {N}")
        n_history = history.numel()
    if (bias_tokens is None) != (cu_bias is None) or (bias_values is None) != (cu_bias is None):
        raise SvwError("bias_tokens, bias_values and cu_bias come together")
    if cu_bias is not None:
        _need_like(gpu, i32, ("bias_tokens", "cu_bias"), (bias_tokens, cu_bias))
        _need_like(gpu, f32, ("bias_values",), (bias_values,))
        n_bias = bias_tokens.numel()
        if cu_bias.numel() != N + 1 or n_bias != bias_values.numel():
            raise SvwError(f"cu_bias must have {N + 1} elements, bias_tokens and bias_values one length")
    if mask is not None:
        _need_like(gpu, i32, ("mask", "mask_row"), (mask, mask_row))
        if mask_row is not None and mask_row.numel() != rows:
            raise SvwError(f"mask_row must have {rows} elements")
        if mask.dim() != 2 or mask.shape[1] != (V + 31) // 32:
            raise SvwError(f"mask must be [mask rows, {(V + 31) // 32}]")
        mask_rows = mask.shape[0]
    elif mask_row is not None:
        raise SvwError("mask_row comes with a mask")
    if out is None:
        out = _empty(stream, gpu, (rows, V), logits.dtype, logits.device)
    elif out is not logits and (out.dtype is not logits.dtype or out.get_device() != gpu or out.shape != logits.shape
                                or out.stride(1) != 1):
        raise SvwError("out must be like logits")
    if workspace is None:
        if need := logits_adjust_workspace_size(N, V, R, n_history, n_bias):
            workspace = _empty(stream, gpu, need, torch.uint8, logits.device, returned=False)
    elif _off(workspace, torch.uint8, gpu):
        raise SvwError(f"workspace must be a contiguous uint8 tensor on cuda:{gpu}")
    # a single row has no pitch of its own
    pitch = logits.stride(0) if rows > 1 else V
    out_pitch = out.stride(0) if rows > 1 else V
    rc = lib().logits_adjust(logits.data_ptr(), pitch, code, V, N, cu_draft.data_ptr(), R, 1 if has_bonus else 0,
                             _addr(draft_tokens), _addr(history), _addr(cu_history), n_history, _addr(prompt_len),
                             _addr(repetition), _addr(frequency), _addr(presence), _addr(bias_tokens),
                             _addr(bias_values), _addr(cu_bias), n_bias, _addr(mask), mask_rows, _addr(mask_row),
                             out.data_ptr(), out_pitch, _addr(status), _addr(workspace),
                             0 if workspace is None else workspace.numel(), _stream_of(stream, gpu))
    if rc:
        _check(rc)
    return out


# svw_paged_kv, field by field; its end is padded as a C struct's is
_pack_paged = struct.Struct("@2P6qPq5i0q").pack


def _paged(k_cache, v_cache, block_table, N):
    """The svw_paged_kv of two [n_pages, heads, page_size, head_dim] tensors
    (any strides but the last) and their block table, their GPU and shape."""
    shape, gpu = k_cache.shape, k_cache.get_device()
    if len(shape) != 4 or v_cache.shape != shape or k_cache.dtype is not v_cache.dtype:
        raise SvwError("k_cache and v_cache must be alike: [n_pages, heads, page_size, head_dim]")
    k0, k1, k2, k3 = k_cache.stride()
    v0, v1, v2, v3 = v_cache.stride()
    if gpu < 0 or v_cache.get_device() != gpu or k3 != 1 or v3 != 1:
        raise SvwError("the caches must be CUDA tensors with contiguous head vectors")
    if block_table.dtype is not _torch().int32 or block_table.get_device() != gpu or block_table.dim() != 2:
        raise SvwError(f"block_table must be an int32 [{N}, max_pages] CUDA tensor")
    rows, mp = block_table.shape
    t0, t1 = block_table.stride()
    if rows != N or (mp > 1 and t1 != 1):
        raise SvwError(f"block_table must be [{N}, max_pages] with contiguous rows")
    pages, heads, size, dim = shape
    return _pack_paged(k_cache.data_ptr(), v_cache.data_ptr(), k0, k1, k2, v0, v1, v2, block_table.data_ptr(),
                       t0 if N > 1 else mp, mp, pages, size, heads, dim), gpu, shape


def _heads(name, t, dim, dtype, gpu):
    """The strides of tokens and heads of a [new tokens, heads, head_dim] tensor."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != dim or stride[2] != 1 or t.dtype is not dtype or t.get_device() != gpu:
        raise SvwError(f"{name} must be [new tokens, heads, {dim}], of the cache's type and GPU, with contiguous heads")
    return shape, stride


def kv_append(k, v, k_cache, v_cache, block_table, cu_new, kv_len, *, cos_sin=None, interleaved: bool = False,
              positions=None, q=None, q_out=None, status=None, stream=None):
    """The new tokens' keys, rotated by their positions, and values written to
    the paged cache.  Returns their rotated queries (None without q).

    k, v: [total_new, heads, head_dim], q: [total_new, query heads, head_dim],
    strided as a split of one projection's output is; k_cache, v_cache:
    [n_pages, heads, page_size, head_dim], any strides (a cache of tokens of
    heads is passed transposed); block_table: int32 [N, max_pages]; cu_new:
    int32 [N + 1]; kv_len: int32 [N], the new tokens counted; cos_sin: float32
    [max_pos, rot_dim], cosines then sines (None: no rotation).  Request i's new
    token t is written at place kv_len[i] - n_i + t and rotated by that
    position, or by positions (int32 [total_new]).
    """
    torch = _torch()
    i32 = torch.int32
    N = cu_new.numel() - 1
    cache, gpu, shape = _paged(k_cache, v_cache, block_table, N)
    _need_current(stream, gpu)
    dim, dtype = shape[3], k_cache.dtype
    kh, ks = _heads("k", k, dim, dtype, gpu)
    vh, vs = _heads("v", v, dim, dtype, gpu)
    T = kh[0]
    if kh[1] != shape[1] or vh != kh:
        raise SvwError("k and v must have the cache's heads and one length")
    if _off(cu_new, i32, gpu) or _off(kv_len, i32, gpu) or _off(positions, i32, gpu) or _off(status, i32, gpu):
        _need_like(gpu, i32, ("cu_new", "kv_len", "positions", "status"), (cu_new, kv_len, positions, status))
    if kv_len.numel() != N:
        raise SvwError(f"kv_len must have {N} elements")
    if positions is not None and positions.numel() != T:
        raise SvwError(f"positions must have {T} elements")
    max_pos = rot = 0
    if cos_sin is not None:
        if _off(cos_sin, torch.float32, gpu) or cos_sin.dim() != 2:
            raise SvwError(f"cos_sin must be a contiguous float32 [max_pos, rot_dim] tensor on cuda:{gpu}")
        max_pos, rot = cos_sin.shape
    hq, qs = 0, (0, 0)
    if q is not None:
        qh, qs = _heads("q", q, dim, dtype, gpu)
        hq = qh[1]
        if qh[0] != T:
            raise SvwError("q must have as many tokens as k")
        if q_out is None:
            q_out = _empty(stream, gpu, qh, dtype, q.device)
        elif _off(q_out, dtype, gpu) or q_out.shape != qh:
            raise SvwError("q_out must be like q, contiguous")
    elif q_out is not None:
        raise SvwError("q_out comes with q")
    rc = lib().kv_append(k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], _addr(q), qs[0], qs[1], _addr(q_out),
                         _dtype_code(k_cache), hq, N, cu_new.data_ptr(), T, kv_len.data_ptr(), _addr(positions),
                         _addr(cos_sin), max_pos, rot, 1 if interleaved else 0, cache, _addr(status),
                         _stream_of(stream, gpu))
    if rc:
        _check(rc)
    return q_out


@functools.lru_cache(maxsize=64)
def paged_attention_workspace_size(total_new: int, n_q_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return int(lib().svw_paged_attention_workspace_size(total_new, n_q_heads, n_kv_heads, head_dim))


def paged_attention(q, k_cache, v_cache, block_table, cu_new, kv_len, *, scale: float | None = None,
                    causal: bool = True, window: int = 0, out=None, lse=None, want_lse: bool = True, status=None,
                    workspace=None, stream=None):
    """Attention of each request's new tokens over its cached keys, their own
    included (as kv_append leaves them).  Returns (out, lse): bf16 [total_new,
    query heads, head_dim] and float32 [total_new, query heads] (None without
    want_lse).

    q: bf16 [total_new, query heads, head_dim]; the caches, block_table, cu_new
    and kv_len as for kv_append.  causal=False: a new token sees its whole
    block; window > 0: only the last `window` keys up to its own.  scale
    defaults to head_dim ** -0.5.
    """
    torch = _torch()
    i32 = torch.int32
    N = cu_new.numel() - 1
    cache, gpu, shape = _paged(k_cache, v_cache, block_table, N)
    _need_current(stream, gpu)
    dim, dtype = shape[3], k_cache.dtype
    qh, qs = _heads("q", q, dim, dtype, gpu)
    T, hq, _ = qh
    if _off(cu_new, i32, gpu) or _off(kv_len, i32, gpu) or _off(status, i32, gpu):
        _need_like(gpu, i32, ("cu_new", "kv_len", "status"), (cu_new, kv_len, status))
    if kv_len.numel() != N:
        raise SvwError(f"kv_len must have {N} elements")
    if out is None:
        out = _empty(stream, gpu, qh, dtype, q.device)
    elif _off(out, dtype, gpu) or out.shape != qh:
        raise SvwError("out must be like q, contiguous")
    if lse is None:
        if want_lse:
            lse = _empty(stream, gpu, (T, hq), torch.float32, q.device)
    elif _off(lse, torch.float32, gpu) or lse.numel() != T * hq:
        raise SvwError(f"lse must be a contiguous float32 [{T}, {hq}] tensor on cuda:{gpu}")
    if workspace is None:
        need = paged_attention_workspace_size(T, hq, shape[1], dim)
        workspace = _empty(stream, gpu, max(1, need), torch.uint8, q.device, returned=False)
    elif _off(workspace, torch.uint8, gpu):
        raise SvwError(f"workspace must be a contiguous uint8 tensor on cuda:{gpu}")
    rc = lib().paged_attention(q.data_ptr(), qs[0], qs[1], _dtype_code(q), hq, N, cu_new.data_ptr(), T,
                               kv_len.data_ptr(), cache, float(dim ** -0.5 if scale is None else scale),
                               1 if causal else 0, int(window), out.data_ptr(), _addr(lse), _addr(status),
                               workspace.data_ptr(), workspace.numel(), _stream_of(stream, gpu))
    if rc:
        _check(rc)
    return out, lse
