"""One request batch decoded with drafted tokens, on random weights.

Shows the operators of a speculative step working together, as a serving loop uses them:

1. a small draft model proposes ``k`` tokens per request, one after another; each is drawn by
   ``sampler.Sampler`` and its distribution is kept;
2. the target model takes the last accepted token and the drafted ones in one pass: per layer
   ``KVAppend`` (norm, rotation, append to the paged cache) and ``ChunkAttention``;
3. ``DraftVerifier`` accepts drafted tokens against the target's probabilities and draws one
   more token per request;
4. the caches' lengths go back to what was accepted: refused tokens' slots are written again.

    python examples/speculative_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from constrained_logits_sampling_gb300.sampler import Sampler  # noqa: E402
from constrained_logits_sampling_gb300.speculative import ChunkAttention, DraftVerifier, KVAppend  # noqa: E402


class Decoder:
    """A decoder of random weights over a paged cache: embedding, ``layers`` of attention and a
    gated product, and an LM head.  Its matrix products are torch's.  Decoders of one seed share
    embedding, head and first layers, so one of fewer layers is a draft model for another."""

    def __init__(self, layers, vocab, Hq, Hkv, D, batch, max_len, page=16, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        hidden = Hq * D

        def w(*shape):
            return (torch.randn(*shape, device="cuda", generator=g) * shape[0] ** -0.5).to(dtype)

        self.Hq, self.Hkv, self.D, self.dtype = Hq, Hkv, D, dtype
        self.embed = torch.randn(vocab, hidden, device="cuda", generator=g).to(dtype)
        self.head = (2.0 * torch.randn(hidden, vocab, device="cuda", generator=g) * hidden ** -0.5).to(dtype)
        self.layers = [dict(qkv=w(hidden, (Hq + 2 * Hkv) * D), out=w(hidden, hidden), up=w(hidden, 2 * hidden),
                            down=w(hidden, hidden), q_norm=torch.ones(D, dtype=dtype, device="cuda"),
                            k_norm=torch.ones(D, dtype=dtype, device="cuda")) for _ in range(layers)]
        pages = (max_len + page - 1) // page
        shape = (batch * pages, page, Hkv, D)
        self.caches = [(torch.empty(shape, dtype=dtype, device="cuda"), torch.empty(shape, dtype=dtype, device="cuda"))
                       for _ in range(layers)]
        self.table = torch.randperm(batch * pages, device="cuda", generator=g).to(torch.int32).view(batch, pages)
        f = 10000.0 ** (-torch.arange(D // 2, device="cuda", dtype=torch.float64) / (D // 2))
        a = torch.arange(max_len, device="cuda", dtype=torch.float64)[:, None] * f
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float()
        self.append, self.attend = KVAppend(), ChunkAttention()

    def __call__(self, tokens, cu_new, kv_lens, max_new):
        """Logits (float32) of each of the batch's new tokens; kv_lens counts them."""
        T = tokens.numel()
        x = self.embed[tokens.long()]
        for w, (k_cache, v_cache) in zip(self.layers, self.caches):
            h = torch.nn.functional.rms_norm(x, x.shape[-1:])
            qkv = h @ w["qkv"]
            heads = (self.Hq, self.Hkv, self.Hkv)
            q, k, v = (t.view(T, n, self.D) for n, t in zip(heads, qkv.split([n * self.D for n in heads], 1)))
            q = self.append(q, k, v, k_cache, v_cache, self.table, cu_new, kv_lens, cos_sin=self.cos_sin,
                            q_weight=w["q_norm"], k_weight=w["k_norm"])["q"]
            o = self.attend(q, k_cache, v_cache, self.table, cu_new, kv_lens, max_new=max_new)["out"]
            x = x + o.flatten(1) @ w["out"]
            up, gate = (torch.nn.functional.rms_norm(x, x.shape[-1:]) @ w["up"]).chunk(2, 1)
            x = x + (up * torch.nn.functional.silu(gate)) @ w["down"]
        return (torch.nn.functional.rms_norm(x, x.shape[-1:]) @ self.head).float()


class SpeculativeLoop:
    """The state of a batch: both models' caches, lengths and the last token of each request."""

    def __init__(self, target, draft, vocab, batch, k, temperature=0.7, seed=1):
        self.target, self.draft, self.B, self.k, self.T = target, draft, batch, k, temperature
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.sampler, self.verify = Sampler(batch, vocab), DraftVerifier()
        self.seeds = torch.arange(1, batch + 1, dtype=torch.int64, device="cuda")
        self.temps = torch.full((batch,), temperature, device="cuda")
        self.one = torch.arange(batch + 1, dtype=torch.int32, device="cuda")

    def prefill(self, prompts):
        """Prompts as lists of token ids; the last token of each is left for the first step."""
        n = [len(p) - 1 for p in prompts]
        cu = torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32, device="cuda")
        lens = torch.tensor(n, dtype=torch.int32, device="cuda")
        flat = torch.tensor([t for p in prompts for t in p[:-1]], dtype=torch.int32, device="cuda")
        for model in (self.target, self.draft):
            model(flat, cu, lens, max(n))
        self.lens = lens  # of both caches
        self.last = torch.tensor([p[-1] for p in prompts], dtype=torch.int32, device="cuda")

    def step(self):
        """One step.  Returns the verifier's outputs: ``tokens`` [B, k + 1] and ``accepted``; the
        probabilities and random numbers it used are kept in ``self.used``."""
        B, k = self.B, self.k
        drafted, probs, token = [], [], self.last
        for i in range(k):
            lens = self.lens + (i + 1)
            logits = self.draft(token, self.one, lens, 1)
            token = self.sampler(logits, temperatures=self.temps, seeds=self.seeds,
                                 positions=lens.to(torch.int64))["tokens"]
            drafted.append(token)
            probs.append(torch.softmax(logits / self.T, 1))
        # the draft's cache gets the last drafted token too, in case all are accepted
        self.draft(token, self.one, self.lens + (k + 1), 1)
        x = torch.stack(drafted, 1)
        rows = torch.cat([self.last[:, None], x], 1).reshape(-1)
        logits = self.target(rows, self.one * (k + 1), self.lens + (k + 1), k + 1)
        used = dict(target_probs=torch.softmax(logits / self.T, 1), draft_tokens=x.reshape(-1).contiguous(),
                    cu_draft=self.one * k, u_accept=torch.rand(B * k, device="cuda", generator=self.gen),
                    u_sample=torch.rand(B, device="cuda", generator=self.gen), max_draft=k,
                    draft_probs=torch.stack(probs, 1).view(B * k, -1))
        out = self.verify(**used)
        self.lens = self.lens + 1 + out["accepted"]
        self.last = out["tokens"].gather(1, out["accepted"].long()[:, None])[:, 0].contiguous()
        self.used = used
        return out


def main(steps=12, batch=6, vocab=4000, k=3):
    shape = dict(vocab=vocab, Hq=8, Hkv=2, D=64, batch=batch, max_len=256)
    target = Decoder(layers=2, seed=0, **shape)
    draft = Decoder(layers=1, seed=0, **shape)
    loop = SpeculativeLoop(target, draft, vocab, batch, k)
    loop.prefill([list(range(7 * b + 1, 7 * b + 6 + 3 * b)) for b in range(batch)])
    accepted = 0
    for _ in range(steps):
        out = loop.step()
        assert not out["status"].any()
        accepted += int(out["accepted"].sum())
    print(f"{steps} steps, {batch} requests: {accepted / (steps * batch):.2f} of {k} drafted tokens accepted per step, "
          f"lengths now {loop.lens.tolist()}")


if __name__ == "__main__":
    main()
