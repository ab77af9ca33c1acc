"""Cases for the operators of one speculative-decoding step, with their plain forms.

Three operators, used one after another when drafted tokens are checked against a target:

* ``append``: per-head RMS norm of queries and keys (optional), position rotation, and the
  append of keys and values to a paged cache (``speculative.append_kv``);
* ``attend``: attention of each sequence's newest tokens over its paged cache
  (``speculative.ChunkAttention``);
* ``verify``: acceptance of drafted tokens against the target's probabilities, and one more
  token per request, from given random numbers (``speculative.verify_draft``).

Lengths of a case follow from the case alone (its "lens" number); values follow from the
seed.  Cache slots past a sequence's length hold NaN, as never-written memory may.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
MASS = float(2 ** 40)


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one request generating token by token: latency
        dict(name="append one token", op="append", B=1, n_lo=1, n_hi=1, old_lo=777, old_hi=777, Hq=32, Hkv=8, D=128,
             page=16, dtype="bf16", norm=True, rot=128, interleaved=False, lens=1),
        # 256 requests, three drafted tokens and the last accepted one each (the verify-scale batch)
        dict(name="append verify 256x4", op="append", B=256, n_lo=4, n_hi=4, old_lo=50, old_hi=500, Hq=32, Hkv=8,
             D=128, page=64, dtype="bf16", norm=True, rot=128, interleaved=False, lens=2),
        # prompts taken in chunks, the largest pass of tokens
        dict(name="append chunks 8192", op="append", B=8, n_lo=1024, n_hi=1024, old_lo=0, old_hi=4000, Hq=32, Hkv=8,
             D=128, page=64, dtype="bf16", norm=False, rot=128, interleaved=False, lens=3),
        # ragged mixed batch: idle sequences, odd lengths, half of each head rotated in pairs, odd group
        dict(name="append ragged", op="append", B=61, n_lo=0, n_hi=37, old_lo=0, old_hi=300, Hq=14, Hkv=2, D=64,
             page=16, dtype="f16", norm=False, rot=32, interleaved=True, lens=4),
        # one request generating token by token: latency
        dict(name="attend one token", op="attend", B=1, n_lo=1, n_hi=1, old_lo=776, old_hi=776, Hq=32, Hkv=8, D=128,
             page=16, dtype="bf16", window=0, lens=5),
        # 256 requests x 4 positions over their contexts (the verify-scale batch)
        dict(name="attend verify 256x4", op="attend", B=256, n_lo=4, n_hi=4, old_lo=200, old_hi=4000, Hq=32, Hkv=8,
             D=128, page=64, dtype="bf16", window=0, lens=6),
        # a few very long contexts, few rows: the long axis has to be split
        dict(name="attend long", op="attend", B=3, n_lo=1, n_hi=8, old_lo=60000, old_hi=131000, Hq=16, Hkv=2, D=128,
             page=128, dtype="f16", window=0, lens=7),
        # prompts taken in chunks over what is already cached: bound by the products
        dict(name="attend chunks 2x2048", op="attend", B=2, n_lo=2048, n_hi=2048, old_lo=12000, old_hi=14336, Hq=32,
             Hkv=8, D=128, page=64, dtype="bf16", window=0, lens=8),
        # ragged mixed batch, a window, one key head per query head, idle and fresh sequences
        dict(name="attend ragged window", op="attend", B=19, n_lo=0, n_hi=150, old_lo=0, old_hi=1000, Hq=12, Hkv=12,
             D=64, page=16, dtype="f16", window=256, lens=9),
        # one request, four drafted tokens, the small vocabulary: latency
        dict(name="verify one request", op="verify", B=1, n_lo=4, n_hi=4, V=32000, dtype="f32", draft=True, noise=0.3,
             lens=10),
        # requests with 0 to 7 tokens proposed by lookup (no draft probabilities), rows that start unaligned
        dict(name="verify lookup 64", op="verify", B=64, n_lo=0, n_hi=7, V=50257, dtype="bf16", draft=False, noise=0.3,
             lens=11),
        # the verify-scale batch: 256 requests x (3 drafted + 1)
        dict(name="verify 256x4", op="verify", B=256, n_lo=3, n_hi=3, V=151936, dtype="f32", draft=True, noise=0.6,
             lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "verify"])
    lens = rng.randrange(1 << 30)
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        D = rng.choice([64, 80, 96, 128, 256])
        B = _log(rng, 1, 256)
        # tokens of the pass and cached tokens both stay under the largest listed pass
        n_hi = _log(rng, 1, max(1, 8 * 1024 * 48 * 128 // ((g * Hkv + 2 * Hkv) * D * B)))
        n_hi = min(n_hi, 2048)
        return dict(op=op, B=B, n_lo=rng.choice([0, 1, n_hi]), n_hi=n_hi, old_lo=0, old_hi=_log(rng, 1, 30000 // B + 1),
                    Hq=g * Hkv, Hkv=Hkv, D=D, page=page, dtype=rng.choice(["bf16", "f16"]),
                    norm=rng.random() < 0.5, rot=rng.choice([D, D, D // 2]), interleaved=rng.random() < 0.3, lens=lens)
    if op == "attend":
        D = rng.choice([64, 128])
        if rng.random() < 0.6:  # few new tokens
            B = _log(rng, 1, 256)
            n_hi = _log(rng, 1, 16)
            old = _log(rng, 16, min(131000, 500000 // B))
        else:  # chunks
            B = _log(rng, 1, 16)
            n_hi = _log(rng, 17, 2048)
            old = _log(rng, 1, 14336)
            while B * n_hi * (old + n_hi) * g * Hkv * D > 2 * 2048 * 14000 * 32 * 128:
                B = max(1, B // 2)
                n_hi = max(17, n_hi * 2 // 3)
        return dict(op=op, B=B, n_lo=rng.choice([0, 1, n_hi]), n_hi=n_hi, old_lo=rng.choice([0, old // 2, old]),
                    old_hi=old, Hq=g * Hkv, Hkv=Hkv, D=D, page=page, dtype=rng.choice(["bf16", "f16"]),
                    window=rng.choice([0, 0, _log(rng, 1, 4096)]), lens=lens)
    V = _log(rng, 1000, 151936)
    n_hi = _log(rng, 1, 8)
    B = _log(rng, 1, max(1, min(256, 1024 * 151936 // (V * (n_hi + 1)))))
    return dict(op=op, B=B, n_lo=rng.choice([0, 1, n_hi]), n_hi=n_hi, V=V, dtype=rng.choice(["f32", "bf16"]),
                draft=rng.random() < 0.7, noise=rng.choice([0.1, 0.3, 1.0]), lens=lens)


def _lengths(case):
    """New tokens and tokens already cached of each sequence (of a verification: drafted tokens)."""
    r = random.Random(case["lens"])
    new = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["B"])]
    if not sum(new):
        new[0] = max(1, case["n_hi"])
    old = [r.randint(case["old_lo"], case["old_hi"]) for _ in range(case["B"])] if "old_lo" in case else None
    return new, old


def _visible(case):
    """(row, key) pairs and keys with at least one row, over all sequences, for one head."""
    new, old = _lengths(case)
    w = case["window"]
    pairs = keys = 0
    for n, o in zip(new, old):
        if not n:
            continue
        for p in range(o, o + n):
            pairs += min(p + 1, w) if w else p + 1
        keys += min(o + n, w - 1 + n) if w else o + n
    return pairs, keys


def work(case):
    new, old = _lengths(case)
    T, e = sum(new), SIZE[case["dtype"]]
    if case["op"] == "append":
        el = T * (case["Hq"] + 2 * case["Hkv"]) * case["D"]
        return {"bytes": 2 * el * e + T * case["rot"] * 4, "flops": 8 * el}
    if case["op"] == "attend":
        pairs, keys = _visible(case)
        by = 2 * T * case["Hq"] * case["D"] * e + 2 * keys * case["Hkv"] * case["D"] * e
        return {"bytes": by, "flops": 4 * pairs * case["Hq"] * case["D"]}
    # one target row per request; the draft's row where a token is refused (counted for half of them)
    rows = case["B"] * (1.5 if case["draft"] else 1.0)
    return {"bytes": int(rows * case["V"] * e), "flops": int(4 * rows * case["V"])}


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _offsets(lens):
    return _i32([0] + list(np.cumsum(lens)))


def _pages(case, lens, seed):
    """A table of pages in random order, with spare pages that no sequence has."""
    need = [(x + case["page"] - 1) // case["page"] for x in lens]
    width = max(max(need), 1) + 1
    order = np.random.default_rng(seed).permutation(sum(need) + 3)
    table = np.zeros((case["B"], width), np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return torch.from_numpy(table).cuda(), sum(need) + 3


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "verify":
        _prepare_verify(case, s, g)
    else:
        _prepare_cache(case, s, g, seed)
    if own:
        _prepare_own(case, s)
    return s


def _prepare_cache(case, s, g, seed):
    new, old = _lengths(case)
    lens = [o + n for o, n in zip(old, new)]
    T, Hq, Hkv, D, dt = sum(new), case["Hq"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
    s.update(new=new, lens=lens, cu=_offsets(new), kv_lens=_i32(lens))
    s["table"], pages = _pages(case, lens, seed)
    shape = (pages, case["page"], Hkv, D)
    s["k_cache"] = torch.randn(shape, dtype=dt, device="cuda", generator=g)
    s["v_cache"] = torch.randn(shape, dtype=dt, device="cuda", generator=g)
    if case["op"] == "append":
        # one projection holds queries, keys and values side by side
        x = torch.randn(T, (Hq + 2 * Hkv) * D, dtype=dt, device="cuda", generator=g) * 1.5
        s["q"] = x[:, :Hq * D].view(T, Hq, D)
        s["k"] = x[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        s["v"] = x[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        s["q_w"] = s["k_w"] = None
        if case["norm"]:
            s["q_w"] = (1 + 0.2 * torch.randn(D, device="cuda", generator=g)).to(dt)
            s["k_w"] = (1 + 0.2 * torch.randn(D, device="cuda", generator=g)).to(dt)
        half = case["rot"] // 2
        f = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        a = torch.arange(max(lens) + 1, dtype=torch.float64, device="cuda")[:, None] * f
        s["cos_sin"] = torch.cat([a.cos(), a.sin()], dim=1).float()
        return
    # some heads look sharply at a few keys, some broadly
    sharp = torch.linspace(0.5, 2.0, Hq, device="cuda")[None, :, None]
    s["q"] = (torch.randn(T, Hq, D, device="cuda", generator=g) * sharp).to(dt)
    for b, n in enumerate(lens):  # slots never written
        if n % case["page"]:
            last = int(s["table"][b, n // case["page"]])
            s["k_cache"][last, n % case["page"]:] = float("nan")
            s["v_cache"][last, n % case["page"]:] = float("nan")


def _prepare_verify(case, s, g):
    new, _ = _lengths(case)
    B, V, N, dt = case["B"], case["V"], sum(new), DTYPES[case["dtype"]]
    s.update(new=new, cu=_offsets(new), most=max(case["n_hi"], max(new)))
    own_rows = torch.tensor([i + b for b in range(B) for i in range(sum(new[:b]), sum(new[:b + 1]))],
                            dtype=torch.long, device="cuda")

    def rows(m):
        return torch.randn(m, V, device="cuda", generator=g)

    # heavy-tailed logits: Student's t with three degrees of freedom, as the verify-scale workload has
    z = rows(N + B)
    z *= 3.0 * ((rows(N + B).square_() + rows(N + B).square_() + rows(N + B).square_()) / 3.0).rsqrt_()
    z.clamp_(-40.0, 25.0)
    s["target"] = torch.softmax(z, dim=1).to(dt)
    zd = z[own_rows] + case["noise"] * rows(N)
    q = torch.softmax(zd, dim=1)
    del z, zd
    e = torch.empty(N, V, device="cuda").exponential_(generator=g)
    s["x"] = (q / e).argmax(dim=1).to(torch.int32)
    del e
    s["draft"] = q.to(dt) if case["draft"] else None
    s["u"] = torch.rand(N, device="cuda", generator=g)
    s["u_last"] = torch.rand(B, device="cuda", generator=g)


def _prepare_own(case, s):
    from constrained_logits_sampling_gb300 import speculative as spec
    dt = DTYPES[case["dtype"]]
    if case["op"] == "append":
        s["out"] = {"q": torch.empty(s["q"].shape, dtype=dt, device="cuda"),
                    "status": torch.empty(case["B"], dtype=torch.int32, device="cuda")}
        s["call"] = spec.KVAppend()
        s["args"] = s["call"].make_args(
            s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_lens"],
            cos_sin=s["cos_sin"], interleaved=case["interleaved"], q_weight=s["q_w"], k_weight=s["k_w"], eps=1e-6,
            q_out=s["out"]["q"], row_status=s["out"]["status"])
        s["out"].update(k_cache=s["k_cache"], v_cache=s["v_cache"])
    elif case["op"] == "attend":
        s["out"] = {"out": torch.empty(s["q"].shape, dtype=dt, device="cuda"),
                    "lse": torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda"),
                    "status": torch.empty(case["B"], dtype=torch.int32, device="cuda")}
        s["call"] = spec.ChunkAttention()
        s["args"] = s["call"].make_args(
            s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_lens"], max_new=max(s["new"]),
            window=case["window"], out=s["out"]["out"], lse=s["out"]["lse"], row_status=s["out"]["status"])
    else:
        B = case["B"]
        s["out"] = {"tokens": torch.empty(B, s["most"] + 1, dtype=torch.int32, device="cuda"),
                    "accepted": torch.empty(B, dtype=torch.int32, device="cuda"),
                    "status": torch.empty(B, dtype=torch.int32, device="cuda")}
        s["call"] = spec.DraftVerifier()
        s["args"] = s["call"].make_args(
            s["target"], s["x"], s["cu"], s["u"], s["u_last"], draft_probs=s["draft"], max_draft=s["most"],
            tokens=s["out"]["tokens"], accepted=s["out"]["accepted"], row_status=s["out"]["status"])


# --------------------------------------------------------------------------- one pass

def run(s):
    if own:
        s["call"].apply(s["args"])
        return s["out"]
    return {"append": _plain_append, "attend": _plain_attend, "verify": _plain_verify}[s["case"]["op"]](s)


def _plain_head(x, w, c, sn, rot, interleaved):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + 1e-6) * w.float()
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * c - b * sn
        y[..., 1:rot:2] = b * c + a * sn
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * c - b * sn
        y[..., rot // 2:rot] = b * c + a * sn
    return y


def _plain_append(s):
    case, cu, dt = s["case"], s["cu"].long(), s["q"].dtype
    rot, page = case["rot"], case["page"]
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    pos = s["kv_lens"].long()[b] - (cu[b + 1] - t)
    cs = s["cos_sin"][pos]
    c, sn = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    q = _plain_head(s["q"], s["q_w"], c, sn, rot, case["interleaved"]).to(dt)
    k = _plain_head(s["k"], s["k_w"], c, sn, rot, case["interleaved"]).to(dt)
    where = s["table"].long()[b, pos // page]
    s["k_cache"][where, pos % page] = k
    s["v_cache"][where, pos % page] = s["v"]
    return {"q": q, "status": torch.zeros(case["B"], dtype=torch.int32, device="cuda"),
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    case, q = s["case"], s["q"]
    Hkv, D, page, w = case["Hkv"], case["D"], case["page"], case["window"]
    G = case["Hq"] // Hkv
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], float("-inf"), device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(s["new"], s["lens"])):
        if not n:
            continue
        ids = s["table"][b, :(m + page - 1) // page].long()
        K = s["k_cache"][ids].reshape(-1, Hkv, D)[:m].float()
        Vv = s["v_cache"][ids].reshape(-1, Hkv, D)[:m].float()
        qb = q[at:at + n].float().view(n, Hkv, G, D)
        pos = torch.arange(m - n, m, device="cuda")[:, None]
        key = torch.arange(m, device="cuda")[None, :]
        hide = key > pos
        if w:
            hide = hide | (key <= pos - w)
        hide = hide[:, None, :].expand(n, G, m).reshape(n * G, m)
        step = Hkv if n * G * Hkv * m <= 1 << 27 else 1
        for h in range(0, Hkv, step):
            x = torch.matmul(qb[:, h:h + step].permute(1, 0, 2, 3).reshape(step, n * G, D),
                             K[:, h:h + step].permute(1, 2, 0)) * (1.0 / math.sqrt(D))
            x = x.masked_fill(hide, float("-inf"))
            top = x.amax(dim=-1, keepdim=True)
            e = torch.exp(x - top)
            tot = e.sum(dim=-1, keepdim=True)
            o = torch.matmul(e, Vv[:, h:h + step].permute(1, 0, 2)) / tot
            out[at:at + n].view(n, Hkv, G, D)[:, h:h + step] = o.view(step, n, G, D).permute(1, 0, 2, 3).to(q.dtype)
            lse[at:at + n].view(n, Hkv, G)[:, h:h + step] = (top + tot.log()).view(step, n, G).permute(1, 0, 2)
        at += n
    return {"out": out, "lse": lse, "status": torch.zeros(case["B"], dtype=torch.int32, device="cuda")}


def _plain_verify(s):
    B, cu, x, most = s["case"]["B"], s["cu"].long(), s["x"].long(), s["most"]
    target, draft = s["target"], s["draft"]
    i = torch.arange(x.shape[0], device="cuda")
    r = torch.arange(B, device="cuda")
    b = torch.searchsorted(cu[1:], i, right=True)
    # products of two 32-bit numbers are exact in 64 bits, so the comparison is too
    p = target[i + b, x].double()
    q = draft[i, x].double() if draft is not None else torch.ones_like(p)
    ok = torch.zeros(B, most + 1, dtype=torch.long, device="cuda")
    ok[b, i - cu[b]] = (s["u"].double() * q < p).long()
    acc = ok.cumprod(dim=1).sum(dim=1)
    refused = acc < cu[1:] - cu[:-1]
    at = cu[:-1] + acc
    P = (target[at + r].float() * MASS).long()
    at = at.clamp(max=max(x.shape[0] - 1, 0))
    if draft is not None:
        Q = (draft[at].float() * MASS).long()
        Q *= refused[:, None]
        W = (P - Q).clamp_(min=0)
    else:
        W = P.clone()
        W[r, x[at]] = torch.where(refused, torch.zeros_like(acc), W[r, x[at]])
    W = torch.where((W.sum(dim=1) == 0)[:, None], P, W)
    C = W.cumsum(dim=1)
    tot = C[:, -1]
    u = (s["u_last"] * 2.0 ** 31).long()
    k = u * (tot >> 31) + ((u * (tot & (2 ** 31 - 1))) >> 31)
    last = (C <= k[:, None]).sum(dim=1)
    out = torch.full((B, most + 1), -1, dtype=torch.int32, device="cuda")
    out[b, i - cu[b]] = torch.where(i - cu[b] < acc[b], x, torch.full_like(x, -1)).to(torch.int32)
    out[r, acc] = last.to(torch.int32)
    return {"tokens": out, "accepted": acc.to(torch.int32),
            "status": torch.zeros(B, dtype=torch.int32, device="cuda")}


# --------------------------------------------------------------------------- from the definition, in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "attend": _exact_attend, "verify": _exact_verify}[case["op"]](case, s)


def _exact_append(case, s):
    rot, half, D = case["rot"], case["rot"] // 2, case["D"]
    first = [2 * j for j in range(half)] if case["interleaved"] else list(range(half))
    second = [2 * j + 1 for j in range(half)] if case["interleaved"] else list(range(half, rot))
    rest = list(range(rot, D))
    pos = np.concatenate([np.arange(m - n, m) for n, m in zip(s["new"], s["lens"])])
    seq = np.repeat(np.arange(case["B"]), s["new"])
    cs = s["cos_sin"].double()[torch.from_numpy(pos).cuda()]
    z = torch.complex(cs[:, :half], cs[:, half:])[:, None, :]

    def turn(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + 1e-6) * w.double()
        t = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * z
        y = torch.empty_like(x)
        y[..., first], y[..., second], y[..., rest] = t.real, t.imag, x[..., rest]
        return y

    q, k = turn(s["q"], s["q_w"]), turn(s["k"], s["k_w"])
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    slot = s["table"].cpu().numpy()[seq, pos // case["page"]].astype(np.int64) * case["page"] + pos % case["page"]
    slot = torch.from_numpy(slot).cuda()
    kc.view(-1, case["Hkv"], D)[slot] = k
    vc.view(-1, case["Hkv"], D)[slot] = s["v"].double()
    return {"q": q, "status": torch.zeros(case["B"], dtype=torch.int32), "k_cache": kc, "v_cache": vc}


def _exact_attend(case, s):
    D, G, page, w = case["D"], case["Hq"] // case["Hkv"], case["page"], case["window"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    table = s["table"].cpu().numpy()
    at = 0
    for b in range(case["B"]):
        n, m = s["new"][b], s["lens"][b]
        j = np.arange(m)
        slots = torch.from_numpy(table[b, j // page].astype(np.int64) * page + j % page).cuda()
        j = torch.from_numpy(j).cuda()
        for c in range(0, n, 1024):
            hi = min(n, c + 1024)
            p = torch.arange(m - n + c, m - n + hi, device="cuda")
            seen = j[None, :] <= p[:, None]
            if w:
                seen &= j[None, :] > p[:, None] - w
            for h in range(case["Hkv"]):
                K = s["k_cache"].view(-1, case["Hkv"], D)[slots, h].double()
                V = s["v_cache"].view(-1, case["Hkv"], D)[slots, h].double()
                for a in range(h * G, h * G + G):
                    y = (s["q"][at + c:at + hi, a].double() @ K.T) / math.sqrt(D)
                    y = torch.where(seen, y, torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
                    l = torch.logsumexp(y, dim=1)
                    out[at + c:at + hi, a] = torch.exp(y - l[:, None]) @ V
                    lse[at + c:at + hi, a] = l
        at += n
    return {"out": out, "lse": lse, "status": torch.zeros(case["B"], dtype=torch.int32)}


def _exact_verify(case, s):
    B = case["B"]
    x, u, ul = s["x"].cpu().numpy(), s["u"].double().cpu().numpy(), s["u_last"].double().cpu().numpy()
    tokens = np.full((B, s["most"] + 1), -1, np.int32)
    accepted = np.zeros(B, np.int32)
    at = 0
    for b in range(B):
        n, a = s["new"][b], 0
        while a < n:
            q = float(s["draft"][at + a, x[at + a]]) if s["draft"] is not None else 1.0
            if not u[at + a] * q < float(s["target"][at + b + a, x[at + a]]):
                break
            tokens[b, a] = x[at + a]
            a += 1
        full = np.floor(s["target"][at + b + a].double().cpu().numpy() * MASS).astype(np.int64)
        rest = full.copy()
        if a < n and s["draft"] is not None:
            rest = np.maximum(full - np.floor(s["draft"][at + a].double().cpu().numpy() * MASS).astype(np.int64), 0)
        elif a < n:
            rest[x[at + a]] = 0
        if not rest.any():
            rest = full
        sums = np.cumsum(rest)
        k = int(math.floor(ul[b] * 2.0 ** 31)) * int(sums[-1]) >> 31
        tokens[b, a] = int(np.searchsorted(sums, k, side="right"))
        accepted[b] = a
        at += n
    return {"tokens": torch.from_numpy(tokens), "accepted": torch.from_numpy(accepted),
            "status": torch.zeros(B, dtype=torch.int32)}
