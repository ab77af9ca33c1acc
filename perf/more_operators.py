"""Cases for the operators of a decoding step whose drafted tokens form a tree, with their plain forms.

Five operators, used one after another when each request has drafted several continuations:

* ``plan``: parents of drafted tokens to what each token may see, its position and the rows'
  offsets (``tree.TreePlan``);
* ``attend``: attention of the tree's tokens over the paged cache and over each other by mask
  (``tree.TreeAttention``);
* ``verify``: a walk down the tree that accepts drafted tokens against the target's probabilities,
  and one more token per request, from given random numbers (``tree.TreeVerifier``);
* ``keep``: keys and values of the accepted path moved together in the cache of every layer, and
  the new lengths (``pages.KeepPath``);
* ``pages``: sequences that share pages of the cache: forked, given room for their next token (a
  shared page that is written to is copied first), trimmed again (``pages.PagePool``, ``pages.CopyPages``).

Row layout of a tree step: request b has rows cu_draft[b] + b ..: its last accepted token, then its
drafted tokens.  Lengths and the trees of attention, verification and moves follow from the case alone (its "lens"
number), values from the seed.  Cache slots past a sequence's length hold NaN, as never-written memory may.
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
        # one request with a tree of 63 drafted tokens: latency
        dict(name="attend one tree", op="attend", B=1, n_lo=63, n_hi=63, deep=6, old_lo=1400, old_hi=1400, Hq=32, Hkv=8,
             D=128, page=16, dtype="bf16", window=0, lens=21),
        # 64 requests x up to 32 rows over their contexts: bound by reading the cache
        dict(name="attend 64 trees", op="attend", B=64, n_lo=23, n_hi=31, deep=8, old_lo=200, old_hi=4000, Hq=32,
             Hkv=8, D=128, page=64, dtype="bf16", window=0, lens=22),
        # few requests, wide trees, long contexts, eight query heads a key head: bound by the products
        dict(name="attend wide trees", op="attend", B=4, n_lo=100, n_hi=191, deep=12, old_lo=30000, old_hi=60000, Hq=32,
             Hkv=4, D=128, page=128, dtype="f16", window=0, lens=23),
        # small ragged trees, idle and fresh sequences, a window, three query heads a key head
        dict(name="attend ragged trees", op="attend", B=95, n_lo=0, n_hi=13, deep=4, old_lo=0, old_hi=1500, Hq=12, Hkv=4,
             D=64, page=16, dtype="f16", window=300, lens=24),
        # one request, candidates that are certain of their tokens, the small vocabulary: latency
        dict(name="verify one tree", op="verify", B=1, n_lo=63, n_hi=63, deep=6, V=32000, dtype="f32", draft=False,
             noise=0.3, lens=25),
        # 64 requests whose children were drawn from the draft's distributions
        dict(name="verify 64 sampled trees", op="verify", B=64, n_lo=15, n_hi=31, deep=6, V=151936, dtype="f32",
             draft=True, noise=0.8, lens=26),
        # one request
        dict(name="plan one tree", op="plan", B=1, n_lo=63, n_hi=63, deep=6, window=0, lens=27),
        # 256 requests of all sizes
        dict(name="plan 256 trees", op="plan", B=256, n_lo=0, n_hi=127, deep=20, window=0, lens=28),
        # one request, one layer: latency
        dict(name="keep one path", op="keep", B=1, n_lo=63, n_hi=63, deep=6, old_lo=700, old_hi=700, Hkv=8, D=128,
             page=16, layers=1, dtype="bf16", lens=29),
        # 192 requests, all layers of a small model in one call
        dict(name="keep 192 paths", op="keep", B=192, n_lo=15, n_hi=31, deep=8, old_lo=20, old_hi=200, Hkv=8, D=128,
             page=32, layers=8, dtype="bf16", lens=30),
        # one prompt continued four times
        dict(name="pages one prompt x4", op="pages", prompts=1, forks=4, old_lo=777, old_hi=777, Hkv=8, D=128, page=16,
             layers=1, dtype="bf16", lens=31),
        # 48 cached prompts, four requests each
        dict(name="pages 48 prompts x4", op="pages", prompts=48, forks=4, old_lo=500, old_hi=8000, Hkv=4, D=128, page=64,
             layers=4, dtype="bf16", lens=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "verify", "verify", "plan", "keep", "pages"])
    lens = rng.randrange(1 << 30)
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    deep = rng.randint(1, 12)
    dtype = rng.choice(["bf16", "f16"])
    if op == "attend":
        B, n, D = _log(rng, 1, 256), _log(rng, 1, 191), rng.choice([64, 128])
        while B * n > 4096:
            B, n = max(1, B // 2), max(1, n * 2 // 3)
        old = _log(rng, 1, min(100000, 400000 // B))
        while B * n * old * g * Hkv * D > 4 * 150 * 50000 * 32 * 128:
            old = max(1, old // 2)
        return dict(op=op, B=B, n_lo=rng.choice([0, n // 2, n]), n_hi=n, deep=deep, old_lo=rng.choice([0, old // 2, old]),
                    old_hi=old, Hq=g * Hkv, Hkv=Hkv, D=D, page=page, dtype=dtype,
                    window=rng.choice([0, 0, _log(rng, 1, 4096)]), lens=lens)
    if op == "verify":
        V, n = _log(rng, 1000, 151936), _log(rng, 1, 63)
        B = _log(rng, 1, max(1, min(256, 64 * 24 * 151936 // (V * (n + 1)))))
        return dict(op=op, B=B, n_lo=rng.choice([0, n // 2, n]), n_hi=n, deep=min(deep, 8), V=V,
                    dtype=rng.choice(["f32", "bf16"]), draft=rng.random() < 0.6, noise=rng.choice([0.1, 0.3, 1.0]), lens=lens)
    if op == "plan":
        n = _log(rng, 1, 255)
        return dict(op=op, B=_log(rng, 1, 256), n_lo=rng.choice([0, n // 2, n]), n_hi=n, deep=rng.randint(1, 40),
                    window=rng.choice([0, 0, rng.randint(1, 12)]), lens=lens)
    D, layers = rng.choice([64, 80, 96, 128, 256]), _log(rng, 1, 12)
    if op == "keep":
        B, n = _log(rng, 1, 192), _log(rng, 1, 63)
        while B * layers * Hkv * D > 192 * 8 * 8 * 128:
            layers = max(1, layers // 2)
            B = max(1, B * 3 // 4)
        return dict(op=op, B=B, n_lo=rng.choice([0, n // 2, n]), n_hi=n, deep=deep, old_lo=0, old_hi=_log(rng, 1, 200),
                    Hkv=Hkv, D=D, page=page, layers=layers, dtype=dtype, lens=lens)
    prompts, forks, old = _log(rng, 1, 48), rng.randint(1, 8), _log(rng, 1, 8000)
    while prompts * (old + forks * page) * layers * Hkv * D > 48 * 4500 * 4 * 4 * 128:
        prompts, layers, old = max(1, prompts // 2), max(1, layers - 1), max(1, old * 2 // 3)
    return dict(op=op, prompts=prompts, forks=forks, old_lo=rng.choice([1, old // 2 + 1, old]), old_hi=max(old, old // 2 + 1),
                Hkv=Hkv, D=D, page=page, layers=layers, dtype=dtype, lens=lens)


def _tree(r, n, deep):
    """Parents of n drafted tokens (-1: the last accepted one), no token deeper than `deep`."""
    parents, depth = [], []
    for i in range(n):
        p = r.randint(max(-1, i - 1 - max(2, n // 3)), i - 1)
        while p >= 0 and depth[p] >= deep:
            p = parents[p]
        parents.append(p)
        depth.append(1 if p < 0 else depth[p] + 1)
    return parents


def _depths(parents):
    d = []
    for p in parents:
        d.append(1 if p < 0 else d[p] + 1)
    return d


def _shape(case):
    """Drafted tokens and tokens already cached of each request, and their trees."""
    r = random.Random(case["lens"])
    new = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["B"])]
    if not sum(new):
        new[0] = max(1, case["n_hi"])
    old = [r.randint(case["old_lo"], case["old_hi"]) for _ in range(case["B"])] if "old_lo" in case else [0] * case["B"]
    return new, old, [_tree(r, n, case["deep"]) for n in new]


def _paths(case, trees):
    """For each tree an accepted path: nodes in order, each a child of the one before."""
    r = random.Random(case["lens"] + 1)
    paths = []
    for parents in trees:
        at, path = -1, []
        for i, p in enumerate(parents):
            if p == at and r.random() < 0.6:
                path.append(i)
                at = i
        paths.append(path)
    return paths


def work(case):
    op = case["op"]
    if op == "pages":
        r, e = random.Random(case["lens"]), SIZE[case["dtype"]]
        by = 0
        for _ in range(case["prompts"]):
            n = r.randint(case["old_lo"], case["old_hi"])
            by += case["forks"] * (12 * -(-n // case["page"]) + 4 * (n % case["page"]) * case["Hkv"] * case["D"] * e * case["layers"])
        return {"bytes": by, "flops": by}
    new, old, trees = _shape(case)
    rows = sum(new) + case["B"]
    if op == "plan":
        words = (case["n_hi"] + 32) // 32
        return {"bytes": 4 * sum(new) + 8 * case["B"] + rows * (4 * words + 4), "flops": rows * case["deep"]}
    if op == "verify":
        # the row that the last token is drawn from, and with a draft the draft's
        by = case["B"] * (2 if case["draft"] else 1) * case["V"] * SIZE[case["dtype"]]
        return {"bytes": by, "flops": by}
    e = SIZE[case["dtype"]]
    if op == "keep":
        moved = sum(i != x for path in _paths(case, trees) for i, x in enumerate(path))
        by = 4 * moved * case["Hkv"] * case["D"] * e * case["layers"]
        return {"bytes": by + 12 * case["B"], "flops": by}
    pairs = keys = 0
    w = case["window"]
    for o, parents in zip(old, trees):
        depth = [0] + _depths(parents)
        pairs += sum(min(o + d + 1, w) if w else o + d + 1 for d in depth)
        keys += (min(o, w - 1) if w else o) + len(depth)
    by = 2 * rows * case["Hq"] * case["D"] * e + 2 * keys * case["Hkv"] * case["D"] * e + 4 * rows * case["Hq"]
    return {"bytes": by, "flops": 4 * pairs * case["Hq"] * case["D"]}


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _offsets(lens):
    return _i32([0] + list(np.cumsum(lens)))


def _pages(page, lens, seed):
    """A table of pages in random order, with spare pages that no sequence has."""
    need = [(x + page - 1) // page for x in lens]
    width = max(max(need), 1) + 1
    order = np.random.default_rng(seed).permutation(sum(need) + 3)
    table = np.zeros((len(lens), width), np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return torch.from_numpy(table).cuda(), sum(need) + 3


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    {"attend": _prepare_attend, "verify": _prepare_verify, "plan": _prepare_plan, "keep": _prepare_keep,
     "pages": _prepare_pages}[case["op"]](case, s, g, seed)
    if own:
        _prepare_own(case, s)
    return s


def _mask(trees, words):
    """Which of its sequence's new tokens each row sees: itself and the tokens it continues."""
    rows = []
    for parents in trees:
        seen = [1]
        for i, p in enumerate(parents):
            seen.append(seen[p + 1] | 1 << (i + 1))
        rows += seen
    m = np.zeros((len(rows), words), np.uint32)
    for i, bits in enumerate(rows):
        for w in range(words):
            m[i, w] = bits >> (32 * w) & 0xffffffff
    return m


def _prepare_attend(case, s, g, seed):
    drafted, old, trees = _shape(case)
    new = [n + 1 for n in drafted]
    lens = [o + n for o, n in zip(old, new)]
    T, Hq, Hkv, D, dt = sum(new), case["Hq"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
    s.update(new=new, lens=lens, cu=_offsets(new), kv_lens=_i32(lens))
    s["mask"] = torch.from_numpy(_mask(trees, (max(new) + 31) // 32).view(np.int32)).cuda()
    s["positions"] = _i32([o + d for o, t in zip(old, trees) for d in [0] + _depths(t)])
    s["table"], pages = _pages(case["page"], lens, seed)
    shape = (pages, case["page"], Hkv, D)
    s["k_cache"] = torch.randn(shape, dtype=dt, device="cuda", generator=g)
    s["v_cache"] = torch.randn(shape, dtype=dt, device="cuda", generator=g)
    # some heads look sharply at a few keys, some broadly
    sharp = torch.linspace(0.5, 2.0, Hq, device="cuda")[None, :, None]
    s["q"] = (torch.randn(T, Hq, D, device="cuda", generator=g) * sharp).to(dt)
    for b, n in enumerate(lens):  # slots never written
        if n % case["page"]:
            last = int(s["table"][b, n // case["page"]])
            s["k_cache"][last, n % case["page"]:] = float("nan")
            s["v_cache"][last, n % case["page"]:] = float("nan")


def _prepare_verify(case, s, g, seed):
    new, _, trees = _shape(case)
    B, V, N, dt = case["B"], case["V"], sum(new), DTYPES[case["dtype"]]
    s.update(new=new, cu=_offsets(new), most=max(new), parents=_i32([p for t in trees for p in t]))

    def rows(m):
        return torch.randn(m, V, device="cuda", generator=g)

    # heavy-tailed logits: Student's t with three degrees of freedom, as the verify-scale workload has
    z = rows(N + B)
    z *= 3.0 * ((rows(N + B).square_() + rows(N + B).square_() + rows(N + B).square_()) / 3.0).rsqrt_()
    z.clamp_(-40.0, 25.0)
    s["target"] = torch.softmax(z, dim=1).to(dt)
    # one row of the draft for each token that has been continued; a drafted token's is its parent's
    first = np.cumsum([0] + new)
    parent_row = [int(first[b]) + b + p + 1 for b, t in enumerate(trees) for p in t]
    wanted = sorted(set(parent_row))
    of = {r: i for i, r in enumerate(wanted)}
    s["draft_rows"] = _i32([of[r] for r in parent_row])
    q = z[torch.tensor(wanted, dtype=torch.long, device="cuda")]
    del z
    q += case["noise"] * rows(len(wanted))
    q = torch.softmax(q, dim=1)
    own_row = s["draft_rows"].long()
    if case["draft"]:  # children drawn independently
        e = torch.empty(N, V, device="cuda").exponential_(generator=g)
        s["x"] = (q[own_row] / e).argmax(dim=1).to(torch.int32) if N else _i32([])
        del e
        s["draft"] = q.to(dt)
    else:  # the k-th child of a token is the draft's k-th choice
        count, order = {}, []
        for r in parent_row:
            order.append(count.get(r, 0))
            count[r] = order[-1] + 1
        top = torch.topk(q, max(order, default=0) + 1, dim=1).indices if N else None
        s["x"] = top[own_row, torch.tensor(order, dtype=torch.long, device="cuda")].to(torch.int32) if N else _i32([])
        s["draft"], s["draft_rows"] = None, None
    s["u"] = torch.rand(N, device="cuda", generator=g)
    s["u_last"] = torch.rand(B, device="cuda", generator=g)


def _prepare_plan(case, s, g, seed):
    new, _, _ = _shape(case)
    r = random.Random(seed)
    trees = [_tree(r, n, case["deep"]) for n in new]
    s.update(new=new, cu=_offsets(new), most=case["n_hi"] + 1, parents=_i32([p for t in trees for p in t]),
             kv_lens=_i32([r.randint(0, 4000) + n + 1 for n in new]))


def _cache(case, pages, g):
    shape = (case["layers"], pages, case["page"], case["Hkv"], case["D"])
    return [torch.randn(shape, dtype=DTYPES[case["dtype"]], device="cuda", generator=g) for _ in range(2)]


def _prepare_keep(case, s, g, seed):
    new, old, trees = _shape(case)
    paths = _paths(case, trees)
    lens = [o + n + 1 for o, n in zip(old, new)]
    s.update(cu=_offsets(new), kv_lens=_i32(lens), accepted=_i32([len(p) for p in paths]))
    width = max(max(len(p) for p in paths), 1)
    s["path"] = _i32([p + [-1] * (width - len(p)) for p in paths])
    s["table"], pages = _pages(case["page"], lens, seed)
    s["k_cache"], s["v_cache"] = _cache(case, pages, g)


def _prepare_pages(case, s, g, seed):
    r = random.Random(case["lens"])
    P, F, page = case["prompts"], case["forks"], case["page"]
    lens = [r.randint(case["old_lo"], case["old_hi"]) for _ in range(P)]
    table, have = _pages(page, lens, seed)
    need = [(x + page - 1) // page for x in lens]
    pages = have + 2 * P * F
    order = torch.from_numpy(np.random.default_rng(seed + 1).permutation(pages).astype(np.int32)).cuda()
    width, B = table.shape[1] + 1, P * (F + 1)
    # rows 0 .. P - 1 are cached prompts, the others idle
    s["table"] = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    held = torch.arange(table.shape[1], device="cuda")[None, :] < _i32(need)[:, None]
    s["table"][:P, :width - 1] = torch.where(held, order[table.long()], torch.full_like(table, -1))
    s["held"] = _i32(need + [0] * (P * F))
    s["kv_lens"] = _i32(lens + [0] * (P * F))
    s["before"] = s["kv_lens"].clone()
    s["new"] = _i32([0] * P + [1] * (P * F))
    s["src"] = torch.arange(P, dtype=torch.int32, device="cuda").repeat_interleave(F)
    s["dst"] = torch.arange(P, B, dtype=torch.int32, device="cuda")
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
    s["refs"][s["table"][:P, :width - 1][held].long()] = 1
    s["k_cache"], s["v_cache"] = _cache(case, pages, g)


def _prepare_own(case, s):
    from constrained_logits_sampling_gb300 import pages, tree
    op, B = case["op"], case.get("B", 0)

    def i32(*shape):
        return torch.empty(shape, dtype=torch.int32, device="cuda")

    if op == "attend":
        s["out"] = {"out": torch.empty_like(s["q"]), "lse": torch.empty(s["q"].shape[:2], device="cuda"), "status": i32(B)}
        s["call"] = tree.TreeAttention()
        s["args"] = s["call"].make_args(
            s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_lens"], mask=s["mask"],
            positions=s["positions"], max_new=max(s["new"]), window=case["window"], out=s["out"]["out"],
            lse=s["out"]["lse"], row_status=s["out"]["status"])
    elif op == "verify":
        s["out"] = {"tokens": i32(B, s["most"] + 1), "path": i32(B, s["most"]), "accepted": i32(B), "status": i32(B)}
        s["call"] = tree.TreeVerifier()
        s["args"] = s["call"].make_args(
            s["target"], s["x"], s["parents"], s["cu"], s["u"], s["u_last"], draft_probs=s["draft"],
            draft_rows=s["draft_rows"], max_draft=s["most"], tokens=s["out"]["tokens"], path=s["out"]["path"],
            accepted=s["out"]["accepted"], row_status=s["out"]["status"])
    elif op == "plan":
        rows = sum(s["new"]) + B
        s["out"] = {"mask": i32(rows, (s["most"] + 31) // 32), "positions": i32(rows), "cu_new": i32(B + 1), "status": i32(B)}
        s["call"] = tree.TreePlan()
        s["args"] = s["call"].make_args(
            s["parents"], s["cu"], s["kv_lens"], max_draft=s["most"] - 1, window=case["window"], mask=s["out"]["mask"],
            positions=s["out"]["positions"], cu_new=s["out"]["cu_new"], row_status=s["out"]["status"])
    elif op == "keep":
        s["out"] = {"kv_lens": i32(B), "status": i32(B)}
        s["call"] = pages.KeepPath()
        s["args"] = s["call"].make_args(
            s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_lens"], s["path"], s["accepted"],
            new_lens=s["out"]["kv_lens"], row_status=s["out"]["status"])
        s["out"].update(k_cache=s["k_cache"], v_cache=s["v_cache"])
    else:
        B = s["held"].numel()
        s["pool"], s["copier"] = pages.PagePool(s["refs"].numel(), case["page"]), pages.CopyPages()
        s["pool"].load(s["refs"])
        made = {"copies": i32(B, 3), "reserve_status": i32(B), "fork_status": i32(s["src"].numel()), "trim_status": i32(B)}
        state = (s["table"], s["held"], s["kv_lens"])
        s["args"] = [
            (s["pool"], s["pool"].fork_args(*state, s["src"], s["dst"], row_status=made["fork_status"])),
            (s["pool"], s["pool"].reserve_args(*state, s["new"], copies=made["copies"], row_status=made["reserve_status"])),
            (s["copier"], s["copier"].make_args(s["k_cache"], s["v_cache"], made["copies"])),
            (s["pool"], s["pool"].trim_args(s["table"], s["held"], s["before"], row_status=made["trim_status"]))]
        s["out"] = dict(made, table=s["table"], held=s["held"], kv_lens=s["kv_lens"], refs=s["pool"].refs,
                        k_cache=s["k_cache"], v_cache=s["v_cache"])


# --------------------------------------------------------------------------- one pass

def run(s):
    if own:
        if s["case"]["op"] == "pages":
            for call, args in s["args"]:
                call.apply(args)
        else:
            s["call"].apply(s["args"])
        return s["out"]
    return {"attend": _plain_attend, "verify": _plain_verify, "plan": _plain_plan, "keep": _plain_keep,
            "pages": _plain_pages}[s["case"]["op"]](s)


def _ok(n):
    return torch.zeros(n, dtype=torch.int32, device="cuda")


def _plain_plan(s):
    cu, n, w = s["cu"].long(), s["most"], s["case"]["window"]
    B = s["case"]["B"]
    i = torch.arange(s["parents"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:], i, right=True)
    at = i - cu[b] + 1
    # a token's step to the one it continues; squaring doubles how far it sees
    sees = torch.eye(n, device="cuda").repeat(B, 1, 1)
    sees[b, at, s["parents"].long() + 1] = 1.0
    reach = 1
    while reach < n:
        sees = (torch.matmul(sees, sees) > 0).float()
        reach *= 2
    depth = sees.sum(dim=2) - 1
    if w:
        sees = sees * (depth[:, :, None] - depth[:, None, :] < w)
    words = (n + 31) // 32
    bits = torch.zeros(B, n, words * 32, dtype=torch.long, device="cuda")
    bits[:, :, :n] = sees.long()
    packed = (bits.view(B, n, words, 32) << torch.arange(32, device="cuda")).sum(dim=3)
    counts = cu[1:] - cu[:-1] + 1
    live = torch.arange(n, device="cuda")[None, :] < counts[:, None]
    first = s["kv_lens"].long() - counts
    return {"mask": packed[live].to(torch.int32), "positions": (first[:, None] + depth.long())[live].to(torch.int32),
            "cu_new": (cu + torch.arange(B + 1, device="cuda")).to(torch.int32), "status": _ok(B)}


def _plain_attend(s):
    case, q = s["case"], s["q"]
    Hkv, D, page, w = case["Hkv"], case["D"], case["page"], case["window"]
    G = case["Hq"] // Hkv
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], float("-inf"), device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(s["new"], s["lens"])):
        ids = s["table"][b, :(m + page - 1) // page].long()
        K = s["k_cache"][ids].reshape(-1, Hkv, D)[:m].float()
        Vv = s["v_cache"][ids].reshape(-1, Hkv, D)[:m].float()
        qb = q[at:at + n].float().view(n, Hkv, G, D)
        key = torch.arange(m, device="cuda")
        j = (key - (m - n)).clamp(min=0)
        hide = (s["mask"][at:at + n].long()[:, j // 32] >> (j % 32) & 1) == 0
        hide = hide & (key >= m - n)
        if w:
            hide = hide | ((key < m - n) & (key <= s["positions"][at:at + n].long()[:, None] - w))
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
    return {"out": out, "lse": lse, "status": _ok(case["B"])}


def _plain_verify(s):
    B, cu, x, most = s["case"]["B"], s["cu"].long(), s["x"].long(), s["most"]
    target, draft, parents = s["target"], s["draft"], s["parents"].long()
    N, dev = x.shape[0], "cuda"
    r = torch.arange(B, device=dev)
    n = cu[1:] - cu[:-1]
    node = torch.full((B,), -1, dtype=torch.long, device=dev)  # the last accepted token
    acc = torch.zeros(B, dtype=torch.long, device=dev)
    share = torch.ones(B, device=dev)   # what is left of the target's mass at the node
    taken = torch.zeros(B, device=dev)  # how often the draft's row has been taken from it
    row = torch.full((B,), -1, dtype=torch.long, device=dev)
    # of a draft that is certain: refused siblings, and the integers of their mass
    gone = torch.zeros(B, target.shape[1], dtype=torch.bool, device=dev) if draft is None else None
    removed = torch.zeros(B, dtype=torch.long, device=dev)
    out = torch.full((B, most + 1), -1, dtype=torch.int32, device=dev)
    path = torch.full((B, most), -1, dtype=torch.int32, device=dev)

    def left():
        """The weights that are left at the node: integers."""
        P = (target[cu[:-1] + r + node + 1].float() * MASS).long()
        if draft is None:
            return P.masked_fill(gone, 0)
        y = draft[row.clamp(min=0)].float() * taken[:, None]
        # (where y is past the target nothing is left, and its integer may not fit)
        return (P - (y.clamp(max=2.0) * MASS).long()).clamp_(min=0)

    for i in range(most):
        at = (cu[:-1] + i).clamp(max=max(N - 1, 0))
        tried = (i < n) & (parents[at] == node)
        t = x[at]
        p = target[cu[:-1] + r + node + 1, t].float()
        if draft is None:
            q, here, rest = share, p.double(), ~gone[r, t]
        else:
            y = draft[s["draft_rows"].long()[at], t].float()
            q = y * share
            mass = ((p * MASS).long() - ((y * taken).clamp(max=2.0) * MASS).long()).clamp(min=0)
            # the first child is compared with the probability itself
            here = torch.where(taken == 0, p.double(), mass.double() / MASS)
            rest = torch.ones_like(tried)
        # products of two 32-bit numbers are exact in 64 bits, so the comparison is too
        ok = tried & rest & (s["u"][at].double() * q.double() < here)
        no = tried & ~ok
        out[r, acc] = torch.where(ok, t, out[r, acc].long()).to(torch.int32)
        path[r, acc.clamp(max=most - 1)] = torch.where(ok, i, path[r, acc.clamp(max=most - 1)].long()).to(torch.int32)
        acc = acc + ok
        node = torch.where(ok, i, node)
        if draft is None:
            removed = torch.where(ok, torch.zeros_like(removed), removed + (p * MASS).long() * (no & rest))
            share = (int(MASS) - removed).clamp(min=0).float() * (1.0 / MASS)
            gone = gone & ~ok[:, None]
            gone[r, t] |= no
        else:
            taken = torch.where(ok, torch.zeros_like(taken), torch.where(no, taken + share, taken))
            row = torch.where(ok, torch.full_like(row, -1), torch.where(no, s["draft_rows"].long()[at], row))
            now = (left().sum(dim=1).float() * (1.0 / MASS)).clamp(max=1.0)
            share = torch.where(ok, torch.ones_like(share), torch.where(no, now, share))
    W = left()
    full = (target[cu[:-1] + r + node + 1].float() * MASS).long()
    W = torch.where((W.sum(dim=1) == 0)[:, None], full, W)
    C = W.cumsum(dim=1)
    tot = C[:, -1]
    u = (s["u_last"] * 2.0 ** 31).long()
    k = u * (tot >> 31) + ((u * (tot & (2 ** 31 - 1))) >> 31)
    out[r, acc] = (C <= k[:, None]).sum(dim=1).to(torch.int32)
    return {"tokens": out, "path": path, "accepted": acc.to(torch.int32), "status": _ok(B)}


def _plain_keep(s):
    case, page = s["case"], s["case"]["page"]
    acc, path, table = s["accepted"].long(), s["path"].long(), s["table"].long()
    root = s["kv_lens"].long() - (s["cu"][1:] - s["cu"][:-1]).long() - 1  # the last accepted token's position
    i = torch.arange(path.shape[1], device="cuda")
    live = i[None, :] < acc[:, None]
    zero = torch.zeros((), dtype=torch.long, device="cuda")
    # (places past a path: the root onto itself)
    src = (root[:, None] + torch.where(live, path + 1, zero)).reshape(-1)
    dst = (root[:, None] + torch.where(live, i[None, :] + 1, zero)).reshape(-1)
    b = torch.arange(case["B"], device="cuda").repeat_interleave(path.shape[1])
    for c in (s["k_cache"], s["v_cache"]):
        rows = c[:, table[b, src // page], src % page]
        c[:, table[b, dst // page], dst % page] = rows
    return {"kv_lens": (root + 1 + acc).to(torch.int32), "status": _ok(case["B"]), "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


def _plain_pages(s):
    page, table, held, lens, refs = s["case"]["page"], s["table"], s["held"], s["kv_lens"], s["refs"]
    B, width = table.shape
    j = torch.arange(width, device="cuda")[None, :]
    pages = refs.shape[0]
    ids = torch.arange(pages, device="cuda")

    def count(where):
        """How often each page is named at these places of the table (a place past the last for none)."""
        at = torch.where(where, table.long(), torch.full_like(table, pages).long()).reshape(-1)
        return torch.zeros(pages + 1, dtype=torch.int32, device="cuda").scatter_add_(
            0, at, torch.ones_like(at, dtype=torch.int32))[:pages]

    # fork: the children's rows are their prompts'
    src, dst = s["src"].long(), s["dst"].long()
    have = (lens[src].long() + page - 1) // page
    shared = j < have[:, None]
    table[dst] = torch.where(shared, table[src], table[dst])
    held[dst], lens[dst] = have.to(torch.int32), lens[src]
    where = torch.zeros(B, width, dtype=torch.bool, device="cuda")
    where[dst] = shared
    refs += count(where)
    # reserve: pages that are missing, and pages of their own where shared ones would be written to
    first, last = (lens.long() // page)[:, None], ((lens + s["new"]).long() - 1) // page
    grows = (s["new"] > 0)[:, None]
    writes = grows & (j >= first) & (j <= last[:, None]) & (j < held[:, None])
    writers = count(writes)
    b = torch.arange(B, device="cuda")[:, None].expand(B, width)
    at = torch.where(writes, table.long(), torch.full_like(table, pages).long())
    final = torch.full((pages + 1,), -1, dtype=torch.long, device="cuda").scatter_reduce_(
        0, at.reshape(-1), b.reshape(-1), "amax")[:pages]
    of = table.long().clamp(min=0)
    keeps = (refs[of] == writers[of]) & (final[of] == b)  # the last of those who write to it, if nobody else has it
    cow = writes & (refs[of] > 1) & ~keeps
    takes = cow | (grows & (j >= held[:, None]) & (j <= last[:, None]))
    rank = torch.cumsum(takes.reshape(-1), 0).view(B, width) - 1
    free = refs == 0
    order = torch.zeros(pages + 1, dtype=torch.long, device="cuda").scatter_(
        0, torch.where(free, torch.cumsum(free, 0) - 1, torch.full_like(ids, pages)), ids)
    given = order[rank.clamp(min=0, max=pages)]
    partial = cow & (j == first) & (lens.long() % page > 0)[:, None]
    any_copy = partial.any(dim=1)
    old_page = torch.where(partial, table.long(), torch.zeros_like(given)).sum(dim=1)
    new_page = torch.where(partial, given, torch.zeros_like(given)).sum(dim=1)
    none = torch.full_like(old_page, -1)
    copies = torch.stack([torch.where(any_copy, old_page, none), torch.where(any_copy, new_page, none),
                          torch.where(any_copy, lens.long() % page, torch.zeros_like(none))], 1).to(torch.int32)
    refs -= count(cow)
    table.copy_(torch.where(takes, given, table.long()).to(torch.int32))
    refs += count(takes)
    held.copy_(torch.where(grows[:, 0], torch.maximum(held.long(), last + 1), held.long()).to(torch.int32))
    # copies
    slot = torch.arange(page, device="cuda")[None, :].expand(B, page)
    live = slot < copies[:, 2:3]
    to, frm, sl = (x[live] for x in (copies[:, 1:2].long().expand(B, page), copies[:, 0:1].long().expand(B, page), slot))
    for c in (s["k_cache"], s["v_cache"]):
        c[:, to, sl] = c[:, frm, sl]
    # trim: back to the prompts
    drops = (j >= ((s["before"].long() + page - 1) // page)[:, None]) & (j < held[:, None])
    refs -= count(drops)
    table.masked_fill_(drops, -1)
    held.copy_(torch.minimum(held.long(), (s["before"].long() + page - 1) // page).to(torch.int32))
    return {"copies": copies, "reserve_status": _ok(B), "fork_status": _ok(src.numel()), "trim_status": _ok(B),
            "table": table, "held": held, "kv_lens": lens, "refs": refs, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# --------------------------------------------------------------------------- from the definition, in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"attend": _exact_attend, "verify": _exact_verify, "plan": _exact_plan, "keep": _exact_keep,
            "pages": _exact_pages}[case["op"]](case, s)


def _none(n):
    return torch.zeros(n, dtype=torch.int32)


def _exact_plan(case, s):
    cu, par, lens = s["cu"].tolist(), s["parents"].tolist(), s["kv_lens"].tolist()
    words, mask, pos = (s["most"] + 31) // 32, [], []
    for b in range(case["B"]):
        n = cu[b + 1] - cu[b]
        for i in range(-1, n):
            bits, steps, at = 0, 0, i
            while True:
                if not case["window"] or steps < case["window"]:
                    bits |= 1 << (at + 1)
                if at < 0:
                    break
                at, steps = par[cu[b] + at], steps + 1
            mask.append([bits >> (32 * w) & 0xffffffff for w in range(words)])
            pos.append(lens[b] - n - 1 + steps)
    return {"mask": torch.from_numpy(np.array(mask, np.uint32).view(np.int32).reshape(-1, words)),
            "positions": torch.tensor(pos, dtype=torch.int32),
            "cu_new": torch.tensor([c + b for b, c in enumerate(cu)], dtype=torch.int32), "status": _none(case["B"])}


def _exact_attend(case, s):
    D, G, page, w = case["D"], case["Hq"] // case["Hkv"], case["page"], case["window"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    table, mask, pos = s["table"].cpu().numpy(), s["mask"].cpu().numpy().view(np.uint32), s["positions"].cpu().numpy()
    at = 0
    for b in range(case["B"]):
        n, m = s["new"][b], s["lens"][b]
        j = np.arange(m)
        slots = torch.from_numpy(table[b, j // page].astype(np.int64) * page + j % page).cuda()
        seen = np.ones((n, m), bool)
        if w:
            seen &= j[None, :] > pos[at:at + n, None] - w
        tail = np.unpackbits(mask[at:at + n].view(np.uint8), axis=1, bitorder="little")
        seen[:, m - n:] = tail[:, :n] != 0
        seen = torch.from_numpy(seen).cuda()
        for h in range(case["Hkv"]):
            K = s["k_cache"].view(-1, case["Hkv"], D)[slots, h].double()
            V = s["v_cache"].view(-1, case["Hkv"], D)[slots, h].double()
            for a in range(h * G, h * G + G):
                y = (s["q"][at:at + n, a].double() @ K.T) / math.sqrt(D)
                y = torch.where(seen, y, torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
                l = torch.logsumexp(y, dim=1)
                out[at:at + n, a] = torch.exp(y - l[:, None]) @ V
                lse[at:at + n, a] = l
        at += n
    return {"out": out, "lse": lse, "status": _none(case["B"])}


def _exact_verify(case, s):
    B, most = case["B"], s["most"]
    x, par, cu = s["x"].tolist(), s["parents"].tolist(), s["cu"].tolist()
    u, ul = s["u"].double().tolist(), s["u_last"].double().tolist()
    rows = s["draft_rows"].tolist() if s["draft"] is not None else None
    tokens, path = np.full((B, most + 1), -1, np.int32), np.full((B, most), -1, np.int32)
    accepted = np.zeros(B, np.int32)
    f32, ones = np.float32, 2 ** 40

    def whole(row):
        return np.floor(row.double().cpu().numpy() * MASS).astype(np.int64)

    for b in range(B):
        node, a = -1, 0
        p = s["target"][cu[b] + b].float()
        full = rest = None      # the target's integers, and what refusals have left of them
        share, taken, mass = f32(1), f32(0), ones
        for i in range(cu[b + 1] - cu[b]):
            k = cu[b] + i
            if par[k] != node:
                continue
            pt = float(p[x[k]])
            if rows is None:
                ok = u[k] * float(share) < pt and (rest is None or rest[x[k]] >= 0)
            else:
                y = f32(float(s["draft"][rows[k], x[k]]))
                ok = u[k] * float(f32(y * share)) < (pt if rest is None else rest[x[k]] / MASS)
            if ok:
                tokens[b, a], path[b, a] = x[k], i
                node, a, rest = i, a + 1, None
                p = s["target"][cu[b] + b + i + 1].float()
                share, taken, mass = f32(1), f32(0), ones
                continue
            if rest is None:
                full = whole(p)
                rest = full.copy()
            if rows is None:
                mass -= max(int(rest[x[k]]), 0)
                rest[x[k]] = -1
                share = f32(max(mass, 0) / MASS)
            else:
                taken = f32(taken + share)
                cut = (s["draft"][rows[k]].float().cpu().numpy() * taken).astype(f32)
                rest = np.maximum(full - np.floor(np.minimum(cut, f32(2)).astype(np.float64) * MASS).astype(np.int64), 0)
                share = min(f32(int(rest.sum())) * f32(2.0 ** -40), f32(1))
        w = whole(p) if rest is None else np.maximum(rest, 0)
        if not w.any():
            w = full
        sums = np.cumsum(w)
        k = int(math.floor(ul[b] * 2.0 ** 31)) * int(sums[-1]) >> 31
        tokens[b, a] = int(np.searchsorted(sums, k, side="right"))
        accepted[b] = a
    return {"tokens": torch.from_numpy(tokens), "path": torch.from_numpy(path), "accepted": torch.from_numpy(accepted),
            "status": _none(B)}


def _exact_keep(case, s):
    kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
    cu, lens, acc, path, table = (s[k].tolist() for k in ("cu", "kv_lens", "accepted", "path", "table"))
    page, new_lens = case["page"], []
    for b in range(case["B"]):
        root = lens[b] - (cu[b + 1] - cu[b]) - 1
        for i in range(acc[b]):
            f, t = root + 1 + path[b][i], root + 1 + i
            for c, was in ((kc, s["k_cache"]), (vc, s["v_cache"])):
                c[:, table[b][t // page], t % page] = was[:, table[b][f // page], f % page]
        new_lens.append(root + 1 + acc[b])
    return {"kv_lens": torch.tensor(new_lens, dtype=torch.int32), "status": _none(case["B"]), "k_cache": kc.float(),
            "v_cache": vc.float()}


def _exact_pages(case, s):
    page, table, refs = case["page"], s["table"].tolist(), s["refs"].tolist()
    held, lens, new = s["held"].tolist(), s["kv_lens"].tolist(), s["new"].tolist()
    kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
    B = len(held)
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        held[b], lens[b] = -(-lens[a] // page), lens[a]
        for i in range(held[b]):
            table[b][i] = table[a][i]
            refs[table[a][i]] += 1
    free = [p for p, r in enumerate(refs) if r == 0]  # before the call: pages are taken from the lowest on
    copies, at = [], 0
    for b in range(B):
        copy = [-1, -1, 0]
        for i in range(lens[b] // page, -(-(lens[b] + new[b]) // page) if new[b] else 0):
            if i < held[b] and refs[table[b][i]] == 1:
                continue
            if i < held[b]:
                refs[table[b][i]] -= 1
                if i * page < lens[b]:
                    copy = [table[b][i], free[at], lens[b] - i * page]
            table[b][i] = free[at]
            refs[free[at]], held[b], at = 1, max(held[b], i + 1), at + 1
        copies.append(copy)
    for f, t, n in copies:
        if n:
            kc[:, t, :n], vc[:, t, :n] = kc[:, f, :n], vc[:, f, :n]
    before = s["before"].tolist()
    for b in range(B):
        for i in range(-(-before[b] // page), held[b]):
            refs[table[b][i]] -= 1
            table[b][i] = -1
        held[b] = min(held[b], -(-before[b] // page))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"copies": i32(copies), "reserve_status": _none(B), "fork_status": _none(len(s["src"])), "trim_status": _none(B),
            "table": i32(table), "held": i32(held), "kv_lens": i32(lens), "refs": i32(refs), "k_cache": kc.float(),
            "v_cache": vc.float()}
