"""A bounded wait of a verification round's steps runs out, without a GPU fault: the
call returns, the status word says so, and the same call afterwards gives the
bits it gave before (svw_set_fault and svw_set_wait_limit, as in
test_gpu_timeout)."""
import numpy as np
import pytest

from test_gpu_timeout import _assert_recovered, _hooks, _run_three  # noqa: F401 (an autouse fixture)

pytestmark = pytest.mark.gpu


def _fp32(ts):
    return [t.float() for t in ts]


def _attend_inputs(new, kv, hq, hkv, d, page=64):
    import torch
    g = torch.Generator(device="cuda").manual_seed(sum(kv))
    pages = [-(-n // page) for n in kv]
    first = np.concatenate([[0], np.cumsum(pages)])
    table = torch.zeros(len(kv), max(pages), dtype=torch.int32)
    for i, n in enumerate(pages):
        table[i, :n] = torch.arange(first[i], first[i + 1], dtype=torch.int32)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    shape = (int(first[-1]), hkv, page, d)
    return (r(sum(new), hq, d), r(*shape), r(*shape), table.cuda(), i32(np.concatenate([[0], np.cumsum(new)])), i32(kv))


@pytest.mark.parametrize("new,kv,d", [
    ([1], [20000], 128), ([1], [20000], 64),                        # joined by the last worker
    ([1] * 40, [3000] * 40, 128), ([1] * 40, [3000] * 40, 64),      # joined by a kernel of its own
    ([300], [2000], 128), ([300], [2000], 64)])                     # row tiles in pairs
def test_attend_values_do_not_come(new, kv, d):
    """The products of every second worker wait for values that are not loaded,
    their scores already under way."""
    import serving_vocab_wide_gb300 as svw
    args = _attend_inputs(new, kv, 8, 2, d)
    _assert_recovered(*_run_three(lambda st: _fp32(svw.paged_attention(*args, status=st))))


@pytest.mark.parametrize("new,kv,d", [([1], [20000], 128), ([1] * 5, [700, 1, 9000, 64, 30000], 64)])
def test_attend_a_warp_does_not_come_to_the_join(new, kv, d):
    """Where the last worker joins, a warp that has given up does not leave the
    other three of its worker at a barrier: they go with it."""
    import serving_vocab_wide_gb300 as svw
    args = _attend_inputs(new, kv, 8, 2, d)
    _assert_recovered(*_run_three(lambda st: _fp32(svw.paged_attention(*args, status=st))))


@pytest.mark.parametrize("V,dtype", [(20488, "bf16"), (20489, "fp32")])
def test_adjust_rows_do_not_come(V, dtype):
    """A CTA whose rows do not reach shared memory stops at the first of them."""
    import serving_vocab_wide_gb300 as svw
    import torch
    n, each = 150, 4
    R = n * each
    assert svw.logits_adjust_workspace_size(n, V, R, 0, 0) > 0
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(R + n, V, generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    cu = torch.arange(0, R + 1, each, dtype=torch.int32, device="cuda")
    tokens = torch.randint(0, V, (R,), generator=g, device="cuda", dtype=torch.int32)
    rep = 1 + torch.rand(n, generator=g, device="cuda")
    call = lambda st: _fp32([svw.logits_adjust(x, cu, tokens, repetition=rep, total_draft_rows=R, status=st)])
    _assert_recovered(*_run_three(call))
