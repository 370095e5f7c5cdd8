"""A bounded wait of paged_attention_fp8 runs out, without a GPU fault: the call
returns, the status word says so, and the same call afterwards gives the bits it
gave before (as test_gpu_round_timeout has it of paged_attention)."""
import pytest

from test_gpu_round_timeout import _attend_inputs, _fp32
from test_gpu_timeout import _assert_recovered, _hooks, _run_three  # noqa: F401 (an autouse fixture)

pytestmark = pytest.mark.gpu


def _call(new, kv, d):
    import serving_vocab_wide_gb300 as svw
    import torch
    q, k, v, *rest = _attend_inputs(new, kv, 8, 2, d)
    k, v = (x.to(torch.float8_e4m3fn) for x in (k, v))
    return lambda st: _fp32(svw.paged_attention_fp8(q, k, v, *rest, status=st))


@pytest.mark.parametrize("new,kv,d", [
    ([1], [20000], 128), ([1], [20000], 64),                        # joined by the last worker
    ([1] * 40, [3000] * 40, 128), ([1] * 40, [3000] * 40, 64),      # joined by a kernel of its own
    ([300], [2000], 128), ([300], [2000], 64)])                     # row tiles in pairs
def test_values_do_not_come(new, kv, d):
    _assert_recovered(*_run_three(_call(new, kv, d)))


@pytest.mark.parametrize("new,kv,d", [([1], [20000], 128), ([1] * 5, [700, 1, 9000, 64, 30000], 64)])
def test_a_warp_does_not_come_to_the_join(new, kv, d):
    _assert_recovered(*_run_three(_call(new, kv, d)))
