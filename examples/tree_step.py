"""One request batch decoded with trees of drafted tokens, on random weights, over a pool of pages.

Shows the operators of a tree step working together, as a serving loop uses them:

1. a prompt is prefilled once and forked for each request (``PagePool.fork``): the requests share its
   pages until they write to them;
2. a small draft model is asked once for each request's most probable tokens, level by level, and
   proposes ``width`` children of the root and ``width`` of the best of each level: a tree, certain of
   its tokens;
3. pages for the step's rows are reserved, and shared ones that they would write to are copied
   (``PagePool.reserve``, ``CopyPages``);
4. the target takes root and tree in one pass: ``TreePlan`` once, per layer ``KVAppend`` by position and
   ``TreeAttention`` by mask;
5. ``TreeVerifier`` accepts a path and draws one more token, ``KeepPath`` moves the path's keys and values
   together in all layers and gives the new lengths, and pages that the refused tokens needed go back
   (``PagePool.trim``).

    python examples/tree_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from constrained_logits_sampling_gb300.pages import CopyPages, KeepPath, PagePool  # noqa: E402
from constrained_logits_sampling_gb300.speculative import ChunkAttention, KVAppend  # noqa: E402
from constrained_logits_sampling_gb300.tree import TreeAttention, TreePlan, TreeVerifier  # noqa: E402


class TreeDecoder:
    """A decoder of random weights over a paged cache of all its layers: embedding, ``layers`` of
    attention and a gated product, and an LM head.  Its matrix products are torch's.  Decoders of one seed
    share embedding, head and first layers, so one of fewer layers is a draft model for another."""

    def __init__(self, layers, vocab, Hq, Hkv, D, pages, max_len, page=16, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        hidden = Hq * D

        def w(*shape):
            return (torch.randn(*shape, device="cuda", generator=g) * shape[0] ** -0.5).to(dtype)

        self.Hq, self.Hkv, self.D, self.dtype = Hq, Hkv, D, dtype
        self.embed = torch.randn(vocab, hidden, device="cuda", generator=g).to(dtype)
        self.head = (2.0 * torch.randn(hidden, vocab, device="cuda", generator=g) * hidden ** -0.5).to(dtype)
        self.layers = [dict(qkv=w(hidden, (Hq + 2 * Hkv) * D), out=w(hidden, hidden), up=w(hidden, 2 * hidden),
                            down=w(hidden, hidden), norm=torch.ones(D, dtype=dtype, device="cuda"))
                       for _ in range(layers)]
        shape = (layers, pages, page, Hkv, D)
        self.k_cache, self.v_cache = (torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(2))
        f = 10000.0 ** (-torch.arange(D // 2, device="cuda", dtype=torch.float64) / (D // 2))
        a = torch.arange(max_len, device="cuda", dtype=torch.float64)[:, None] * f
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float()
        self.append, self.chunk, self.tree = KVAppend(), ChunkAttention(), TreeAttention()

    def __call__(self, tokens, table, cu_new, kv_lens, max_new, plan=None):
        """Logits (float32) of each of the batch's new tokens; kv_lens counts them.  ``plan``: of a tree."""
        T = tokens.numel()
        x = self.embed[tokens.long()]
        for w, k_cache, v_cache in zip(self.layers, self.k_cache, self.v_cache):
            qkv = torch.nn.functional.rms_norm(x, x.shape[-1:]) @ w["qkv"]
            heads = (self.Hq, self.Hkv, self.Hkv)
            q, k, v = (t.view(T, n, self.D) for n, t in zip(heads, qkv.split([n * self.D for n in heads], 1)))
            q = self.append(q, k, v, k_cache, v_cache, table, cu_new, kv_lens, cos_sin=self.cos_sin, q_weight=w["norm"],
                            k_weight=w["norm"], positions=plan and plan["positions"])["q"]
            if plan is None:
                o = self.chunk(q, k_cache, v_cache, table, cu_new, kv_lens, max_new=max_new)["out"]
            else:
                o = self.tree(q, k_cache, v_cache, table, cu_new, kv_lens, mask=plan["mask"], max_new=max_new)["out"]
            x = x + o.flatten(1) @ w["out"]
            up, gate = (torch.nn.functional.rms_norm(x, x.shape[-1:]) @ w["up"]).chunk(2, 1)
            x = x + (up * torch.nn.functional.silu(gate)) @ w["down"]
        return (torch.nn.functional.rms_norm(x, x.shape[-1:]) @ self.head).float()


class Cache:
    """One model's pool of pages and the batch's tables, held pages and lengths."""

    def __init__(self, model, batch, max_len, page=16):
        self.model, self.pool = model, PagePool(model.k_cache.shape[1], page)
        self.table = torch.full((batch, -(-max_len // page)), -1, dtype=torch.int32, device="cuda")
        self.held, self.lens = (torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(2))
        self.copy = CopyPages()

    def reserve(self, new):
        """Room for ``new`` tokens of each sequence, its own."""
        got = self.pool.reserve(self.table, self.held, self.lens, new)
        self.copy(self.model.k_cache, self.model.v_cache, got["copies"])
        return got["status"]

    def fork(self, src, dst):
        return self.pool.fork(self.table, self.held, self.lens, src, dst)

    def trim(self):
        return self.pool.trim(self.table, self.held, self.lens)


class TreeLoop:
    """A batch of requests that continue one prompt.  Row 0 of the tables is the prompt itself."""

    def __init__(self, target, draft, batch, max_len, width=3, depth=3, temperature=0.7, seed=1):
        self.B, self.width, self.depth, self.T = batch, width, depth, temperature
        self.target, self.draft = Cache(target, batch + 1, max_len), Cache(draft, batch + 1, max_len)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.plan, self.verify, self.keep = TreePlan(), TreeVerifier(), KeepPath()
        # level d has `width` children of the first token of the level before (the root first)
        parents = [-1 if d == 0 else (d - 1) * width for d in range(depth) for _ in range(width)]
        self.n = len(parents)
        self.parents = torch.tensor(parents * batch, dtype=torch.int32, device="cuda")
        self.rows = torch.arange(batch + 1, dtype=torch.int32, device="cuda")

    def prefill(self, prompt):
        """A list of token ids; the last one is left for the first step of every request."""
        n = len(prompt) - 1
        new = torch.zeros(self.B + 1, dtype=torch.int32, device="cuda")
        new[0] = n
        flat = torch.tensor(prompt[:-1], dtype=torch.int32, device="cuda")
        everybody = self.rows[1:].contiguous()
        for c in (self.target, self.draft):
            bad = c.reserve(new).any()
            c.lens[0] = n
            if n:
                c.model(flat, c.table[:1].contiguous(), torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                        c.lens[:1].contiguous(), n)
            assert not bad and not c.fork(torch.zeros_like(everybody), everybody).any()
        self.last = torch.full((self.B,), prompt[-1], dtype=torch.int32, device="cuda")

    def _draft(self):
        """Drafted tokens [B, n]: the most probable ones of each level."""
        c, one = self.draft, self.rows
        new = torch.full((self.B + 1,), self.depth, dtype=torch.int32, device="cuda")
        new[0] = 0
        assert not c.reserve(new).any()
        token, levels = self.last, []
        lens = c.lens[1:].clone()
        for _ in range(self.depth):
            lens = lens + 1
            logits = c.model(token, c.table[1:], one, lens, 1)
            levels.append(torch.topk(logits, self.width, dim=1).indices.to(torch.int32))
            token = levels[-1][:, 0].contiguous()
        return torch.cat(levels, 1)

    def step(self):
        """One step.  Returns the verifier's outputs; what it was given is kept in ``self.used``."""
        B, n, c = self.B, self.n, self.target
        x = self._draft()
        new = torch.full((B + 1,), n + 1, dtype=torch.int32, device="cuda")
        new[0] = 0
        assert not c.reserve(new).any()
        lens, table = c.lens[1:] + (n + 1), c.table[1:].contiguous()
        cu_draft = self.rows * n
        plan = self.plan(self.parents, cu_draft, lens, max_draft=n)
        rows = torch.cat([self.last[:, None], x], 1).reshape(-1)
        logits = c.model(rows, table, plan["cu_new"], lens, n + 1, plan)
        self.used = dict(target_probs=torch.softmax(logits / self.T, 1), draft_tokens=x.reshape(-1).contiguous(),
                         parents=self.parents, cu_draft=cu_draft, max_draft=n, max_path=self.depth,
                         u_accept=torch.rand(B * n, device="cuda", generator=self.gen),
                         u_sample=torch.rand(B, device="cuda", generator=self.gen))
        out = self.verify(**self.used)
        kept = self.keep(c.model.k_cache, c.model.v_cache, table, cu_draft, lens, out["path"], out["accepted"])
        assert not kept["status"].any()
        c.lens[1:] = kept["kv_lens"]
        assert not c.trim().any()
        # the draft model takes what was kept into its own cache, from the last token that it has
        self._follow(out)
        self.last = out["tokens"].gather(1, out["accepted"].long()[:, None])[:, 0].contiguous()
        return out

    def _follow(self, out):
        c, acc = self.draft, out["accepted"]
        new = torch.zeros(self.B + 1, dtype=torch.int32, device="cuda")
        new[1:] = acc + 1
        assert not c.reserve(new).any()
        rows = torch.cat([self.last[:, None], out["tokens"][:, :self.depth]], 1)
        flat = rows[torch.arange(self.depth + 1, device="cuda")[None, :] <= acc[:, None]].contiguous()
        cu = torch.zeros(self.B + 1, dtype=torch.int32, device="cuda")
        cu[1:] = torch.cumsum(acc + 1, 0)
        c.lens[1:] += acc + 1
        c.model(flat, c.table[1:].contiguous(), cu, c.lens[1:].contiguous(), self.depth + 1)
        assert not c.trim().any()


def main(steps=12, batch=6, vocab=4000):
    shape = dict(vocab=vocab, Hq=8, Hkv=2, D=64, pages=120, max_len=320)
    target, draft = TreeDecoder(layers=2, seed=0, **shape), TreeDecoder(layers=1, seed=0, **shape)
    loop = TreeLoop(target, draft, batch, max_len=320)
    loop.prefill(list(range(3, 60)))
    accepted = 0
    for _ in range(steps):
        out = loop.step()
        assert not out["status"].any()
        accepted += int(out["accepted"].sum())
    free = int((loop.target.pool.refs == 0).sum())
    print(f"{steps} steps, {batch} requests: {accepted / (steps * batch):.2f} of at most {loop.depth} drafted tokens accepted "
          f"per step, lengths now {loop.target.lens.tolist()}, {free} of {loop.target.pool.num_pages} pages free")


if __name__ == "__main__":
    main()
