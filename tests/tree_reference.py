"""Plain references of the operators of a tree step and of a cache's pages, in 64 bits, exact rationals
or plain Python on the CPU.  Shared by the tests; imports nothing of the CUDA path."""
import math
import random
from fractions import Fraction as F

import numpy as np
import torch

import spec_reference as R

F64 = torch.float64


def tree(rng, n, deep=6, wide=3):
    """Parents of n drafted tokens, none deeper than `deep`."""
    parents, depth = [], []
    for i in range(n):
        p = rng.randint(max(-1, i - 1 - wide), i - 1)
        while p >= 0 and depth[p] >= deep:
            p = parents[p]
        parents.append(p)
        depth.append(1 if p < 0 else depth[p] + 1)
    return parents


def chain(n):
    return list(range(-1, n - 1))


def ancestors(parents, window=0):
    """For each row of a request (the root first) the rows it sees and its depth."""
    rows = [([0], 0)]
    for i, p in enumerate(parents):
        at, line = i, [i + 1]
        while parents[at] >= 0:
            at = parents[at]
            line.append(at + 1)
        line.append(0)
        rows.append((line[:window] if window else line, len(line) - 1))
    return rows


def words_of(rows, words):
    """Mask words (as int32) of rows that are lists of numbers."""
    m = np.zeros((len(rows), words), np.uint32)
    for r, seen in enumerate(rows):
        for j in seen:
            m[r, j >> 5] |= np.uint32(1 << (j & 31))
    return torch.from_numpy(m.view(np.int32))


def attention(pr, rows, positions=None, window=0, scale=None):
    """out, lse and bounds of their errors as spec_reference.attention has them; rows: for each row of
    the step the new tokens it sees; positions: where each stands (None: its place)."""
    scale = 1.0 / math.sqrt(pr.D) if scale is None else scale
    u = R.ROUND[pr.dtype]
    out = torch.zeros(pr.T, pr.Hq, pr.D, dtype=F64)
    tol = torch.zeros(pr.T, pr.Hq, pr.D, dtype=F64)
    lse = torch.full((pr.T, pr.Hq), -math.inf, dtype=F64)
    lse_tol = torch.zeros(pr.T, pr.Hq, dtype=F64)
    g, at = pr.Hq // pr.Hkv, 0
    for b in range(pr.B):
        n, m = pr.new[b], pr.lens[b]
        old = m - n
        k, v = pr.seq_kv(b) if n else (None, None)
        for i in range(n):
            t = at + i
            pos = old + i if positions is None else positions[t]
            see = [x for x in range(max(0, pos - window + 1) if window else 0, old)] + sorted(old + j for j in rows[t])
            if not see:
                continue
            for h in range(pr.Hq):
                kk, vv = k[see, h // g], v[see, h // g]
                q = pr.q[t, h].to(F64)
                y = kk @ q * scale
                size = float(((kk.abs() @ q.abs()) * scale).max())
                w = torch.softmax(y, 0)
                out[t, h] = w @ vv
                lse[t, h] = torch.logsumexp(y, 0)
                delta = 2.0 ** -24 * (16 + 8 * size)  # relative error of a weight from its exponent
                tol[t, h] = (u + 2 * delta) * (w @ vv.abs()) + u * out[t, h].abs() + 1e-7
                if pr.dtype == torch.float16:
                    tol[t, h] += 2.0 ** -25 * vv.abs().sum(0) / torch.exp(lse[t, h] - y.max())
                lse_tol[t, h] = delta + 2.0 ** -22 * (1 + abs(float(lse[t, h])))
        at += n
    return out, lse, tol, lse_tol


def f32(x):
    """A rational rounded to float32, to nearest and ties to even, as a rational; exact for what a
    float64 holds, which products of two float32 and integers below 2^53 are."""
    d = float(x)
    assert F(d) == x
    return F(float(np.float32(d)))


ONE = 2 ** 40


def verify_tree(target, draft, rows, x, parents, cu, u, u_last, most):
    """tokens, path and accepted by the rule of include/clsample.h (numpy arrays; probabilities
    float32; draft None or [M, V] with each token's row)."""
    B, V = len(u_last), target.shape[1]
    tokens, path = np.full((B, most + 1), -1, np.int32), np.full((B, most), -1, np.int32)
    accepted = np.zeros(B, np.int32)
    for b in range(B):
        lo, n = int(cu[b]), int(cu[b + 1] - cu[b])
        node, a = -1, 0
        s, c, refused = F(1), F(0), []

        def whole():
            return [math.floor(F(float(p)) * ONE) for p in target[lo + b + node + 1]]

        def left():
            P = whole()
            if draft is None:
                return [0 if t in {int(x[lo + j]) for j in refused} else P[t] for t in range(V)]
            q = draft[rows[lo + refused[-1]]]
            return [max(P[t] - math.floor(f32(F(float(q[t])) * c) * ONE), 0) for t in range(V)]

        for i in range(n):
            if parents[lo + i] != node or a == most:
                continue
            t, p = int(x[lo + i]), F(float(target[lo + b + node + 1, x[lo + i]]))
            ui = F(float(u[lo + i]))
            if draft is None:
                ok = ui * s < p and t not in {int(x[lo + j]) for j in refused}
            else:
                q = F(float(draft[rows[lo + i], t]))
                have = F(left()[t], ONE) if refused else p
                ok = ui * f32(q * s) < have
            if ok:
                tokens[b, a], path[b, a] = t, i
                node, a = i, a + 1
                s, c, refused = F(1), F(0), []
                continue
            refused.append(i)
            if draft is None:
                P = whole()
                s = F(f32(max(ONE - sum(P[t] for t in {int(x[lo + j]) for j in refused}), 0)), ONE)
            else:
                c = F(float(np.float32(float(c)) + np.float32(float(s))))
                s = min(F(f32(sum(left())), ONE), F(1))
        w = left() if refused else whole()
        if not any(w):
            w = whole()
        k = math.floor(F(float(u_last[b])) * 2 ** 31) * sum(w) // 2 ** 31
        run, t = 0, 0
        while True:
            run += w[t]
            if run > k:
                break
            t += 1
        tokens[b, a], accepted[b] = t, a
    return tokens, path, accepted


class Pool:
    """The pool of pages in plain Python, one sequence after another."""

    def __init__(self, pages, page, B, width):
        self.page, self.refs = page, [0] * pages
        self.table = [[-1] * width for _ in range(B)]
        self.held, self.lens, self.B, self.width = [0] * B, [0] * B, B, width

    def need(self, n):
        return -(-n // self.page)

    def fork(self, src, dst):
        status, todo = [], []
        for i, (a, b) in enumerate(zip(src, dst)):
            ok = (0 <= a < self.B and 0 <= b < self.B and b not in src and dst.count(b) == 1 and self.held[b] == 0 and
                  0 <= self.lens[a] <= self.width * self.page and self.need(self.lens[a]) <= self.held[a] <= self.width)
            ok = ok and all(0 <= p < len(self.refs) and self.refs[p] > 0 for p in self.table[a][:self.need(self.lens[a])])
            status.append(0 if ok else 2)
            if ok:
                todo.append((a, b))
        for a, b in todo:
            self.held[b], self.lens[b] = self.need(self.lens[a]), self.lens[a]
            for k in range(self.held[b]):
                self.table[b][k] = self.table[a][k]
                self.refs[self.table[a][k]] += 1
        return status

    def reserve(self, new):
        P, cap = len(self.refs), self.width * self.page
        bad, takes = [], []
        refs = list(self.refs)
        for b in range(self.B):
            n, m, h = new[b], self.lens[b], self.held[b]
            no = n < 0 or m < 0 or m + n > cap or not 0 <= h <= self.width or self.need(m) > h
            span = range(m // self.page, self.need(m + n)) if not no and n else []
            no = no or any(not 0 <= self.table[b][k] < P or self.refs[self.table[b][k]] < 1 for k in span if k < h)
            bad.append(no)
            takes.append([])
            for k in ([] if no else span):
                if k < h:
                    id = self.table[b][k]
                    if refs[id] == 1:
                        continue
                    refs[id] -= 1
                takes[b].append(k)
        free = [p for p in range(P) if self.refs[p] == 0]
        total = sum(len(t) for t in takes)
        copies = [[-1, -1, 0] for _ in range(self.B)]
        if total > len(free):
            return copies, [2 if bad[b] else 1 if takes[b] else 0 for b in range(self.B)], len(free)
        at = 0
        for b in range(self.B):
            for k in takes[b]:
                if k < self.held[b]:
                    old = self.table[b][k]
                    self.refs[old] -= 1
                    if k * self.page < self.lens[b]:
                        copies[b] = [old, free[at], self.lens[b] - k * self.page]
                self.table[b][k] = free[at]
                self.refs[free[at]] = 1
                at += 1
            if not bad[b] and new[b]:
                self.held[b] = max(self.held[b], self.need(self.lens[b] + new[b]))
        return copies, [2 if x else 0 for x in bad], len(free) - total

    def trim(self):
        status = []
        for b in range(self.B):
            m, h = self.lens[b], self.held[b]
            if m < 0 or m > self.width * self.page or not 0 <= h <= self.width or self.need(m) > h:
                status.append(2)
                continue
            ok = True
            for k in range(self.need(m), h):
                id = self.table[b][k]
                self.table[b][k] = -1
                if not 0 <= id < len(self.refs) or self.refs[id] < 1:
                    ok = False
                else:
                    self.refs[id] -= 1
            self.held[b] = self.need(m)
            status.append(0 if ok else 2)
        return status


def rng(seed):
    return random.Random(seed)
