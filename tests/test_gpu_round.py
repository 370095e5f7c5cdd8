"""The steps of verification rounds together, as the example runs them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("seed,lengths", [(1, (5, 40, 17, 130)), (2, (2, 300))])
def test_rounds_emit_the_tokens_of_plain_decoding(seed, lengths):
    """kv_append, paged_attention, logits_adjust (penalties, a ban, a grammar)
    and spec_verify at T = 0: the emitted tokens are those of decoding one by
    one, banned ones and those outside the grammar never among them."""
    import torch
    import serving_vocab_wide_gb300 as svw
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    svw.build()
    spec = importlib.util.spec_from_file_location("verify_round", os.path.join(ROOT, "examples", "verify_round.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    plain, texts, rounds = m.run(seed, lengths)
    assert texts == plain
    assert sum(map(sum, rounds)) > 0, "no draft was accepted"
    for i, (t, n) in enumerate(zip(texts, lengths)):
        assert 4 not in t[n:]
        assert i % 2 or all(tok % 2 == 0 for tok in t[n:])
