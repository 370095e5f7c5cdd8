"""Verification rounds end to end on a toy target model: the steps that precede
spec_verify, as a serving loop would call them.

Each round, for a ragged batch of requests: the last emitted token and the
drafted ones go through the model (kv_append, paged_attention), their logits are
adjusted in place (logits_adjust: penalties, a ban, a grammar) and verified
(spec_verify); the accepted drafts and the verifier's token are emitted.  The
model is one attention layer with random weights.  At temperature 0 the emitted
tokens are those of decoding token by token, which the script also does and
compares.

    python examples/verify_round.py
"""
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import serving_vocab_wide_gb300 as svw  # noqa: E402

V, HIDDEN, HQ, HKV, D, PAGE = 8000, 256, 8, 2, 64, 16


def csr(lens):
    import torch
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), device="cuda")


class Target:
    """One attention layer over a paged cache, and the logits."""

    def __init__(self, seed, requests, longest):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32)
        self.embed = (w(V, HIDDEN) * 0.5).to(torch.bfloat16)
        self.qkv = (w(HIDDEN, (HQ + 2 * HKV) * D) / HIDDEN ** 0.5).to(torch.bfloat16)
        self.out = (w(HQ * D, HIDDEN) / (HQ * D) ** 0.5).to(torch.bfloat16)
        self.head = (w(HIDDEN, V) * 0.5).to(torch.bfloat16)
        pages = -(-longest // PAGE)
        shape = (requests * pages, HKV, PAGE, D)
        self.k_cache = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        self.v_cache = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        self.table = torch.arange(requests * pages, dtype=torch.int32, device="cuda").view(requests, pages)
        inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
        angle = torch.arange(longest, dtype=torch.float64, device="cuda")[:, None] * inv
        self.cos_sin = torch.cat((angle.cos(), angle.sin()), 1).float()

    def __call__(self, tokens, new, kv_len):
        """The logits after each of `tokens` (packed, new[i] of request i, which then has kv_len[i] tokens)."""
        import torch
        x = self.embed[torch.tensor(tokens, device="cuda")]
        q, k, v = (x @ self.qkv).split((HQ * D, HKV * D, HKV * D), 1)
        where = (self.k_cache, self.v_cache, self.table, csr(new),
                 torch.tensor(kv_len, dtype=torch.int32, device="cuda"))
        q = svw.kv_append(k.view(-1, HKV, D), v.view(-1, HKV, D), *where, cos_sin=self.cos_sin, q=q.view(-1, HQ, D))
        o, _ = svw.paged_attention(q, *where)
        return (x + o.view(-1, HQ * D) @ self.out) @ self.head


class Rules:
    """What every request's logits are adjusted by: penalties, a banned token, a
    grammar (even tokens only) for every other request."""

    def __init__(self, requests):
        import torch
        full = lambda v: torch.full((requests,), v, device="cuda")
        self.factors = {"repetition": full(1.2), "frequency": full(0.3), "presence": full(0.2)}
        self.mask = torch.full((1, (V + 31) // 32), 0x55555555, dtype=torch.int32, device="cuda")
        self.bias = {"bias_tokens": torch.full((requests,), 4, dtype=torch.int32, device="cuda"),
                     "bias_values": full(float("-inf")), "cu_bias": csr([1] * requests)}

    def __call__(self, logits, texts, prompts, drafts):
        import torch
        i32 = lambda a: torch.tensor(np.asarray(a, np.int32), device="cuda")
        lens = [len(d) for d in drafts]
        rows = np.repeat([-1 if i % 2 else 0 for i in range(len(texts))], np.add(lens, 1))
        return svw.logits_adjust(logits, csr(lens), i32(sum(drafts, [])), history=i32(sum(texts, [])),
                                 cu_history=csr([len(t) for t in texts]), prompt_len=i32(prompts),
                                 mask=self.mask, mask_row=i32(rows), total_draft_rows=sum(lens), out=logits,
                                 **self.factors, **self.bias)


def start(seed, prompts, longest):
    """The model with the prompts' keys and values cached, all but their last tokens."""
    model = Target(seed, len(prompts), longest)
    model(sum((p[:-1] for p in prompts), []), [len(p) - 1 for p in prompts], [len(p) - 1 for p in prompts])
    return model


def decode(seed, prompts, steps):
    """Greedy decoding, a token per request and step."""
    model, rules = start(seed, prompts, max(map(len, prompts)) + steps + 1), Rules(len(prompts))
    texts = [list(p) for p in prompts]
    for _ in range(steps):
        logits = model([t[-1] for t in texts], [1] * len(texts), [len(t) for t in texts])
        rules(logits, texts, [len(p) for p in prompts], [[] for _ in texts])
        for t, tok in zip(texts, logits.float().argmax(1).tolist()):
            t.append(tok)
    return texts


def speculate(seed, prompts, steps, draft):
    """Verification rounds until every request has `steps` tokens; draft(i, text)
    drafts for request i.  Returns the texts and each round's accepted lengths."""
    import torch
    longest = max(map(len, prompts)) + steps + svw.SVW_MAX_LEN + 2
    model, rules = start(seed, prompts, longest), Rules(len(prompts))
    texts, rounds = [list(p) for p in prompts], []
    while min(len(t) - len(p) for t, p in zip(texts, prompts)) < steps:
        drafts = [draft(i, t) for i, t in enumerate(texts)]
        lens = [len(d) for d in drafts]
        logits = model(sum(([t[-1]] + d for t, d in zip(texts, drafts)), []), [n + 1 for n in lens],
                       [len(t) + n for t, n in zip(texts, lens)])
        rules(logits, texts, [len(p) for p in prompts], drafts)
        tokens = torch.tensor(sum(drafts, []), dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        accepted, emitted = svw.spec_verify(logits, torch.zeros(sum(lens), V, dtype=logits.dtype, device="cuda"),
                                            csr(lens), tokens, 0.0, 0, total_draft_rows=sum(lens), status=status)
        if svw.device_status(int(status)):
            raise RuntimeError("a request was rejected")
        for t, d, a, tok in zip(texts, drafts, accepted.tolist(), emitted.tolist()):
            t += d[:a] + [tok]
        rounds.append(accepted.tolist())
    return [t[:len(p) + steps] for t, p in zip(texts, prompts)], rounds


def run(seed=1, lengths=(5, 40, 17, 130), steps=24):
    """Both ways on the same prompts; drafts are the right tokens, some spoilt."""
    rng = np.random.default_rng(seed)
    prompts = [rng.integers(0, V, n).tolist() for n in lengths]
    plain = decode(seed, prompts, steps + svw.SVW_MAX_LEN)

    def draft(i, text):
        n = int(rng.choice((2, 4, 8, 16)))
        right = plain[i][len(text):len(text) + n]
        right += [0] * (n - len(right))
        return [int(rng.integers(0, V)) if rng.random() < 0.15 else t for t in right]

    texts, rounds = speculate(seed, prompts, steps, draft)
    return [p[:len(t)] for p, t in zip(plain, texts)], texts, rounds


if __name__ == "__main__":
    svw.build()
    plain, texts, rounds = run()
    for n, a in enumerate(rounds):
        print(f"round {n}: accepted {a}")
    print("the same tokens as decoding one by one:", plain == texts)
    sys.exit(0 if plain == texts else 1)
