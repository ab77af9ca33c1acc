"""Plain references of the speculative-step operators, in 64 bits on the CPU, and small
problems for them.  Shared by the tests; imports nothing of the CUDA path."""
import math

import numpy as np
import torch

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # unit roundoff
F64 = torch.float64


class Problem:
    """Sequences with `new[b]` new tokens each and lengths `lens[b]`, over a paged cache whose
    untouched slots hold NaN and whose unused table entries hold invalid ids."""

    def __init__(self, new, lens, Hq, Hkv, D, page, dtype, seed=0, layout="nhd", spare=2):
        g = torch.Generator().manual_seed(seed)
        self.new, self.lens, self.Hq, self.Hkv, self.D, self.page = list(new), list(lens), Hq, Hkv, D, page
        self.dtype, self.B, self.T = dtype, len(new), sum(new)
        need = [(x + page - 1) // page for x in lens]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        self.table = torch.full((self.B, max(need + [1]) + 1), -7, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
            at += m
        self.cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        self.kv_lens = torch.tensor(lens, dtype=torch.int32)
        shape = (self.pages, page, Hkv, D) if layout == "nhd" else (self.pages, Hkv, page, D)
        caches = [torch.full(shape, float("nan")).to(dtype) for _ in range(2)]
        self.k_cache, self.v_cache = (c if layout == "nhd" else c.transpose(1, 2) for c in caches)
        for b, m in enumerate(lens):
            for x in range(m):
                p = int(self.table[b, x // page])
                self.k_cache[p, x % page] = torch.randn(Hkv, D, generator=g).to(dtype)
                self.v_cache[p, x % page] = torch.randn(Hkv, D, generator=g).to(dtype)
        # queries, keys and values as slices of one projection
        fused = torch.randn(self.T, (Hq + 2 * Hkv) * D, generator=g).to(dtype)
        self.q = fused[:, :Hq * D].view(self.T, Hq, D)
        self.k = fused[:, Hq * D:(Hq + Hkv) * D].view(self.T, Hkv, D)
        self.v = fused[:, (Hq + Hkv) * D:].view(self.T, Hkv, D)

    def seq_kv(self, b):
        m = self.lens[b]
        slots = [(int(self.table[b, x // self.page]), x % self.page) for x in range(m)]
        k = torch.zeros(m, self.Hkv, self.D, dtype=F64)
        v = torch.zeros(m, self.Hkv, self.D, dtype=F64)
        for x, (p, s) in enumerate(slots):
            k[x], v[x] = self.k_cache[p, s].to(F64), self.v_cache[p, s].to(F64)
        return k, v


def attention(pr, window=0, scale=None):
    """out, lse, and a bound of the admissible error of each output element: the weights are
    rounded to the type (roundoff u), the result is rounded to it, float32 products and
    exponentials are off by a few units of 2^-24 times the size of the scores, and in float16
    a weight under 2^-14 is off by up to 2^-25."""
    scale = 1.0 / math.sqrt(pr.D) if scale is None else scale
    u = ROUND[pr.dtype]
    out = torch.zeros(pr.T, pr.Hq, pr.D, dtype=F64)
    tol = torch.zeros(pr.T, pr.Hq, pr.D, dtype=F64)
    lse = torch.full((pr.T, pr.Hq), -math.inf, dtype=F64)
    lse_tol = torch.zeros(pr.T, pr.Hq, dtype=F64)
    g = pr.Hq // pr.Hkv
    at = 0
    for b in range(pr.B):
        n, m = pr.new[b], pr.lens[b]
        k, v = pr.seq_kv(b)
        for i in range(n):
            pos = m - n + i
            lo = max(0, pos - window + 1) if window else 0
            if pos < 0:
                continue
            for h in range(pr.Hq):
                kk, vv = k[lo:pos + 1, h // g], v[lo:pos + 1, h // g]
                q = pr.q[at + i, h].to(F64)
                y = kk @ q * scale
                size = float(((kk.abs() @ q.abs()) * scale).max())
                w = torch.softmax(y, 0)
                out[at + i, h] = w @ vv
                lse[at + i, h] = torch.logsumexp(y, 0)
                delta = 2.0 ** -24 * (16 + 8 * size)  # relative error of a weight from its exponent
                mag = w @ vv.abs()
                tol[at + i, h] = (u + 2 * delta) * mag + u * out[at + i, h].abs() + 1e-7
                if pr.dtype == torch.float16:
                    tol[at + i, h] += 2.0 ** -25 * vv.abs().sum(0) / torch.exp(lse[at + i, h] - y.max())
                lse_tol[at + i, h] = delta + 2.0 ** -22 * (1 + abs(float(lse[at + i, h])))
        at += n
    return out, lse, tol, lse_tol


def append(pr, cos_sin=None, rot=0, interleaved=False, q_weight=None, k_weight=None, eps=1e-6):
    """q, caches and the error bound of q and k: one rounding to the type and a few float32
    operations on elements of the row's size."""
    pos = [m - n + i for n, m in zip(pr.new, pr.lens) for i in range(n)]
    seq = [b for b, n in enumerate(pr.new) for _ in range(n)]
    half = rot // 2

    def turn(x, w, t):
        x = x.to(F64)
        if w is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(F64)
        y = x.clone()
        for j in range(half):
            i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            c, s = float(cos_sin[pos[t], j]), float(cos_sin[pos[t], half + j])
            y[:, i0] = x[:, i0] * c - x[:, i1] * s
            y[:, i1] = x[:, i1] * c + x[:, i0] * s
        return y, ROUND[pr.dtype] * y.abs() + 2.0 ** -20 * x.abs().amax(-1, keepdim=True) + 2.0 ** -25

    q, qt = torch.zeros(pr.T, pr.Hq, pr.D, dtype=F64), torch.zeros(pr.T, pr.Hq, pr.D, dtype=F64)
    k, kt = torch.zeros(pr.T, pr.Hkv, pr.D, dtype=F64), torch.zeros(pr.T, pr.Hkv, pr.D, dtype=F64)
    where = []
    for t in range(pr.T):
        q[t], qt[t] = turn(pr.q[t], q_weight, t)
        k[t], kt[t] = turn(pr.k[t], k_weight, t)
        where.append((int(pr.table[seq[t], pos[t] // pr.page]), pos[t] % pr.page) if pos[t] >= 0 else None)
    return q, qt, k, kt, where


def verify(target, draft, x, cu, u, u_last, most):
    """Tokens and accepted counts by the rule of include/clsample.h, in Python integers and
    exact rationals (the inputs are numpy arrays; probabilities float32)."""
    from fractions import Fraction as F
    B, V = len(u_last), target.shape[1]
    tokens = np.full((B, most + 1), -1, np.int32)
    accepted = np.zeros(B, np.int32)
    for b in range(B):
        lo, n, a = int(cu[b]), int(cu[b + 1] - cu[b]), 0
        while a < n:
            q = F(float(draft[lo + a, x[lo + a]])) if draft is not None else F(1)
            if not F(float(u[lo + a])) * q < F(float(target[lo + b + a, x[lo + a]])):
                break
            tokens[b, a] = x[lo + a]
            a += 1
        full = [math.floor(F(float(p)) * 2 ** 40) for p in target[lo + b + a]]
        w = list(full)
        if a < n:
            for t in range(V):
                q = F(float(draft[lo + a, t])) if draft is not None else F(int(t == x[lo + a]))
                w[t] = max(full[t] - math.floor(q * 2 ** 40), 0)
        if not any(w):
            w = full
        k = math.floor(F(float(u_last[b])) * 2 ** 31) * sum(w) // 2 ** 31
        run, t = 0, 0
        while True:
            run += w[t]
            if run > k:
                break
            t += 1
        tokens[b, a] = t
        accepted[b] = a
    return tokens, accepted
