"""The operators of a tree step on the GPU against references in 64 bits and exact rationals
(tree_reference)."""
import math
import random

import numpy as np
import pytest

import spec_reference as R
import tree_reference as TR

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, FP = torch.bfloat16, torch.float16
I32 = torch.int32


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from constrained_logits_sampling_gb300 import build, speculative, tree
    build.build()
    tree.KVAppend, tree.DraftVerifier = speculative.KVAppend, speculative.DraftVerifier
    return tree


def gpu(t):
    """On the device with the strides it has here."""
    if t.dim() == 4 and not t.is_contiguous():
        return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    return t.cuda()


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def offsets(n):
    return i32([0] + list(np.cumsum(n)))


# ----------------------------------------------------------------------------- plan

def run_plan(S, trees, old, most=None, window=0, **kw):
    n = [len(t) for t in trees]
    most = max(n) if most is None else most
    lens = [o + m + 1 for o, m in zip(old, n)]
    got = S.TreePlan()(i32([p for t in trees for p in t]), offsets(n), i32(lens), max_draft=most, window=window, **kw)
    rows = [r for t in trees for r in TR.ancestors(t, window)]
    assert got["status"].tolist() == [0] * len(trees)
    assert torch.equal(got["mask"].cpu(), TR.words_of([r[0] for r in rows], (most + 32) // 32))
    assert got["positions"].tolist() == [o + d for o, t in zip(old, trees) for _, d in TR.ancestors(t)]
    assert got["cu_new"].tolist() == [c + b for b, c in enumerate([0] + list(np.cumsum(n)))]
    return got


@pytest.mark.parametrize("sizes,most,window", [
    ([0], 0, 0), ([1], 1, 0), ([63], 63, 0), ([31, 32, 33, 0, 64], 64, 0), ([5, 1], 200, 0), ([200, 7, 0, 130], 200, 3),
    ([40], 40, 1), ([3] * 700, 3, 0), ([1023, 600], 1023, 0), ([1023], 1023, 40)])
def test_plan(S, sizes, most, window):
    r = random.Random(sum(sizes) + window)
    run_plan(S, [TR.tree(r, n, deep=1 + n % 23, wide=1 + n // 2) for n in sizes], [r.randint(0, 9999) for _ in sizes], most,
             window)


def test_plan_of_chains_and_stars(S):
    run_plan(S, [TR.chain(1023), [-1] * 1023, TR.chain(64), [-1, 0, 0, 0, 1, 1, 1, 4, 4]], [0, 7, 2 ** 30 - 65, 1])


def test_plan_strides_stream_and_graph(S):
    r = random.Random(5)
    trees = [TR.tree(r, n) for n in (20, 0, 45)]
    n = [20, 0, 45]
    parents, cu, lens = i32([p for t in trees for p in t]), offsets(n), i32([30, 9, 99])
    want = S.TreePlan()(parents, cu, lens, max_draft=45)
    wide = torch.full((68, 7), -9, dtype=I32, device="cuda")
    plan = S.TreePlan()
    pos, status = torch.full((68,), -9, dtype=I32, device="cuda"), torch.full((3,), -9, dtype=I32, device="cuda")
    args = plan.make_args(parents, cu, lens, max_draft=45, mask=wide[:, 1:5], positions=pos, row_status=status)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan.apply(args, side)
    torch.cuda.synchronize()
    assert torch.equal(wide[:, 1:3], want["mask"]) and torch.equal(pos, want["positions"])
    assert (wide[:, 0] == -9).all() and (wide[:, 3:] == -9).all()  # two words a row are written
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.apply(args)
    wide.fill_(-9)
    lens += 5
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(wide[:, 1:3], want["mask"]) and torch.equal(pos, want["positions"] + 5)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("kind", ["kernel", "host", "device", "fill", "streams", "first"])
def test_plan_behind_other_work(S, kind, graph):
    """Whatever the work before it is, a call takes what that leaves; the work after it takes the call's."""
    r = random.Random(8)
    trees = [TR.tree(r, n) for n in (20, 0, 45, 63)]
    parents, cu, lens = i32([p for t in trees for p in t]), offsets([len(t) for t in trees]), i32([30, 9, 99, 70])
    if kind == "fill":
        parents.fill_(-1)
    want = S.TreePlan()(parents, cu, lens, max_draft=63)
    host = parents.cpu().pin_memory()
    given, side, plan = torch.empty_like(parents), torch.cuda.Stream(), S.TreePlan()
    out = {n: torch.empty_like(want[n]) for n in ("mask", "positions", "status")}
    copies = {n: torch.empty_like(t) for n, t in out.items()}
    args = plan.make_args(given, cu, lens, max_draft=63, mask=out["mask"], positions=out["positions"],
                          row_status=out["status"])

    def work():
        if kind == "streams":  # behind two of them
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                torch.cuda._sleep(300000)
                given.copy_(parents)
            torch.cuda._sleep(1000)
            torch.cuda.current_stream().wait_stream(side)
        elif kind != "first":
            torch.cuda._sleep(300000)
            if kind == "kernel":
                torch.add(parents, 0, out=given)
            elif kind == "fill":
                given.fill_(-1)
            else:
                given.copy_(host if kind == "host" else parents, non_blocking=True)
        plan.apply(args)
        for n, t in out.items():
            copies[n].copy_(t)

    main = torch.cuda.Stream()
    for _ in range(3):
        given.copy_(parents) if kind == "first" else given.fill_(-7)
        for t in list(out.values()) + list(copies.values()):
            t.fill_(-3)
        torch.cuda.synchronize()
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                work()
            g.replay()
        else:
            with torch.cuda.stream(main):
                work()
        torch.cuda.synchronize()
        for n in out:
            assert torch.equal(copies[n], want[n]), n


def test_plan_bad_requests(S):
    """Requests that cannot be are INVALID with empty masks; the others are what they were."""
    good = [-1, 0, 0]
    parents = good + [-1, 1, 0] + good + [-1, -2, 0] + good + good
    n = [3] * 6
    lens = [10, 10, 3, 10, 2 ** 30 + 1, 4]
    got = S.TreePlan()(i32(parents), offsets(n), i32(lens), max_draft=3)
    assert got["status"].tolist() == [0, 2, 2, 2, 2, 0]
    m = got["mask"].view(6, 4).cpu()
    assert torch.equal(m[0], torch.tensor([1, 3, 7, 11], dtype=I32)) and torch.equal(m[5], m[0])
    assert not m[1:5].any() and not got["positions"].view(6, 4)[1:5].any()
    assert got["positions"].view(6, 4)[5].tolist() == [0, 1, 2, 2]
    # offsets back and past the end: their rows are not written
    got = S.TreePlan()(i32(good * 4), i32([0, 3, 2, 6, 13]), i32([9] * 4), max_draft=4)
    assert got["status"].tolist() == [0, 2, 2, 2]  # the third's first token (the list's third) has itself as parent
    got = S.TreePlan()(i32(good), offsets([3]), i32([9]), max_draft=2)  # more tokens than the bound
    assert got["status"].tolist() == [2] and not got["mask"].any()


# ----------------------------------------------------------------------------- attention

ATTEND = [
    # drafted, old, Hq, Hkv, D, page, dtype, window, layout
    ([0], [0], 4, 4, 64, 16, BF, 0, "nhd"),
    ([0], [776], 32, 8, 128, 16, BF, 0, "nhd"),
    ([3], [0], 4, 1, 64, 16, BF, 0, "nhd"),
    ([3, 3, 3], [5, 60, 300], 8, 2, 128, 16, BF, 0, "hnd"),
    ([7, 0, 15, 2], [64, 63, 1000, 0], 3, 3, 64, 16, FP, 0, "nhd"),  # up to 16 packed rows
    ([2, 1], [4000, 130], 10, 2, 128, 5, BF, 0, "nhd"),  # pages that end inside a tile, odd group
    ([5, 3], [70, 33], 4, 2, 128, 1, FP, 0, "hnd"),
    ([7], [400], 2, 1, 64, 24, BF, 7, "nhd"),  # a window inside the tree's depth
    ([15], [300], 1, 1, 128, 128, FP, 40, "nhd"),
    ([31], [20], 4, 1, 128, 16, BF, 0, "nhd"),  # one row tile
    ([63], [1400], 8, 2, 128, 16, BF, 0, "nhd"),  # two
    ([63], [250], 4, 4, 64, 64, FP, 0, "hnd"),
    ([100, 5, 140], [50, 500, 333], 6, 2, 128, 64, BF, 0, "nhd"),  # three tiles
    ([191], [127], 4, 2, 64, 32, BF, 0, "nhd"),  # the tree over three key tiles
    ([150], [700], 4, 4, 64, 16, FP, 50, "nhd"),
    ([64, 0, 70], [0, 3, 129], 5, 1, 64, 8, BF, 0, "nhd"),
    ([33, 90], [1200, 200], 6, 2, 128, 24, FP, 0, "nhd"),  # pages that are no boxes
    ([40, 33], [129, 2500], 8, 2, 64, 48, BF, 300, "hnd"),
    ([20], [6000], 4, 1, 128, 64, BF, 0, "nhd"),  # a long unit in many parts
    ([25, 30], [2500, 1200], 6, 2, 64, 256, FP, 700, "hnd"),  # pages longer than a tile, a window
    ([19 if i % 40 == 0 else i % 3 for i in range(310)], [(11 * i) % 70 for i in range(310)], 4, 2, 64, 16, BF, 0, "nhd"),
    ([300], [5], 1, 1, 64, 128, BF, 0, "nhd"),
]


def problem(drafted, old, Hq, Hkv, D, page, dtype, layout="nhd", seed=0):
    new = [n + 1 for n in drafted]
    return R.Problem(new, [o + n for o, n in zip(old, new)], Hq, Hkv, D, page, dtype, seed=seed, layout=layout)


def tensors(pr):
    return [pr.q.cuda(), gpu(pr.k_cache), gpu(pr.v_cache), pr.table.cuda(), pr.cu.cuda(), pr.kv_lens.cuda()]


def check_attention(S, pr, rows, positions=None, window=0, handle=None, words=None, ref=None, **kw):
    words = words or (max(pr.new) + 31) // 32
    att = handle or S.TreeAttention()
    out = torch.full((pr.T, pr.Hq, pr.D), 7.0, dtype=pr.dtype, device="cuda")
    got = att(*tensors(pr), mask=TR.words_of(rows, words).cuda(), positions=None if positions is None else i32(positions),
              window=window, max_new=max(pr.new), lse=True, out=out, **kw)
    torch.cuda.synchronize()
    want, lse, tol, lse_tol = ref or TR.attention(pr, rows, positions, window, kw.get("scale"))
    assert got["status"].cpu().tolist() == [0] * pr.B
    assert torch.isfinite(got["out"].float()).all()
    err = (got["out"].cpu().double() - want).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())
    gl = got["lse"].cpu().double()
    assert torch.equal(gl == -math.inf, lse == -math.inf)
    seen = lse > -math.inf
    assert ((gl - lse)[seen].abs() <= lse_tol[seen]).all()
    return got


def trees_of(drafted, seed, window=0):
    r = random.Random(seed)
    trees = [TR.tree(r, n, deep=2 + n % 9, wide=2 + n // 3) for n in drafted]
    lines = [TR.ancestors(t, window) for t in trees]
    return trees, [row[0] for t in lines for row in t], [[row[1] for row in t] for t in lines]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"{c[0][:3]}-{c[1][:3]}-{c[2]}x{c[3]}x{c[4]}-p{c[5]}-w{c[7]}")
def test_attention(S, case):
    drafted, old, Hq, Hkv, D, page, dtype, window, layout = case
    pr = problem(drafted, old, Hq, Hkv, D, page, dtype, layout, seed=len(old) + D)
    _, rows, depth = trees_of(drafted, D + page, window)
    check_attention(S, pr, rows, [o + d for o, t in zip(old, depth) for d in t], window)


@pytest.mark.parametrize("Hkv,G,D,page,dtype", [(3, 1, 128, 16, BF), (5, 2, 64, 12, FP), (7, 1, 64, 64, BF)])
def test_attention_of_many_units(S, Hkv, G, D, page, dtype):
    """So many that key heads go in pairs, of an odd number of them; some sequences have one row or none."""
    B = 6 * torch.cuda.get_device_properties(0).multi_processor_count // Hkv + 1
    drafted = [(70 if i % 80 == 3 else 45) if i % 40 == 3 else i % 2 for i in range(B)]
    old = [(37 * i) % 60 + (400 if i % 160 == 3 else 0) for i in range(B)]
    pr = problem(drafted, old, Hkv * G, Hkv, D, page, dtype, seed=Hkv)
    _, rows, depth = trees_of(drafted, Hkv)
    check_attention(S, pr, rows, [o + d for o, t in zip(old, depth) for d in t])


@pytest.mark.parametrize("n", [17, 33, 64, 65])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("wide", [0, 400])
def test_attention_whatever_the_table_holds(S, n, D, wide):
    """The same results from tables of few and of many pages, which the choice of kernels rests on."""
    pr = problem([n - 1, 0, n // 2], [150, 700, 3], 4, 2, D, 64, BF, seed=n + D)
    _, rows, depth = trees_of([n - 1, 0, n // 2], n)
    if wide:
        pr.table = torch.cat([pr.table, torch.full((3, wide), -1, dtype=I32)], 1)
    check_attention(S, pr, rows, [o + d for o, t in zip((150, 700, 3), depth) for d in t], window=90 if n == 33 else 0)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("drafted,old,Hkv,D", [([3, 9], [700, 90], 2, 64), ([70, 5], [2500, 2000], 8, 128),
                                              ([60 if i % 50 == 1 else i % 3 for i in range(320)], [300] * 320, 2, 128)])
def test_attention_behind_other_work(S, drafted, old, Hkv, D, graph):
    """A call takes what the work before it leaves, of each of its inputs (in one kernel, another, or both)."""
    pr = problem(drafted, old, 4 * Hkv, Hkv, D, 16, BF, seed=6)
    _, rows, depth = trees_of(drafted, 6, 200)
    good = tensors(pr) + [TR.words_of(rows, 3).cuda(), i32([o + d for o, t in zip(old, depth) for d in t])]
    att, kw = S.TreeAttention(), dict(window=200, max_new=max(pr.new))
    want = att(*good[:6], mask=good[6], positions=good[7], lse=True, **kw)
    given = [torch.empty_like(t) for t in good]
    out, status = torch.empty_like(want["out"]), torch.empty_like(want["status"])
    args = att.make_args(*given[:6], mask=given[6], positions=given[7], out=out, row_status=status, **kw)
    seen, ok = torch.empty_like(out), torch.empty_like(status)

    def work(last):
        for i, (t, g) in enumerate(zip(given, good)):
            if i != last:
                t.copy_(g)
        torch.cuda._sleep(300000)
        torch.add(good[last], 0, out=given[last])
        att.apply(args)
        seen.copy_(out)
        ok.copy_(status)

    for last in range(len(good)):
        for t in given:
            t.fill_(-1)
        seen.fill_(7)
        torch.cuda.synchronize()
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                work(last)
            g.replay()
        else:
            work(last)
        torch.cuda.synchronize()
        assert torch.equal(seen, want["out"]) and torch.equal(ok, want["status"]), last


def test_attention_two_handles_at_once(S):
    """Calls of two objects on two streams do not meet."""
    cases = []
    for seed, drafted, old in ((1, [60, 3], [3000, 900]), (2, [100, 30], [2000, 4000])):
        pr = problem(drafted, old, 8, 2, 128, 16, BF, seed=seed)
        _, rows, _ = trees_of(drafted, seed)
        handle = S.TreeAttention()
        alone = check_attention(S, pr, rows, handle=handle)["out"]
        args, mask = tensors(pr), TR.words_of(rows, 4).cuda()
        cases.append((handle, args, mask, max(pr.new), alone, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (handle, args, mask, most, _, stream) in enumerate(cases):
            got[i].append(handle(*args, mask=mask, max_new=most, stream=stream)["out"])
    torch.cuda.synchronize()
    for i, case in enumerate(cases):
        assert all(torch.equal(o, case[4]) for o in got[i])


def test_attention_takes_the_plan(S):
    drafted, old = [30, 0, 17], [100, 7, 640]
    pr = problem(drafted, old, 8, 2, 64, 16, BF, seed=3)
    trees, rows, depth = trees_of(drafted, 3)
    plan = run_plan(S, trees, old)
    assert torch.equal(plan["mask"].cpu(), TR.words_of(rows, 1))
    q, k, v, table, _, lens = tensors(pr)
    got = S.TreeAttention()(q, k, v, table, plan["cu_new"], lens, mask=plan["mask"], positions=plan["positions"], max_new=31)
    want, _, tol, _ = TR.attention(pr, rows)
    assert ((got["out"].cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("n,old,G,D,page", [(4, 37, 4, 64, 16), (13, 0, 1, 128, 8), (40, 100, 3, 64, 16), (90, 0, 2, 128, 24),
                                            (70, 250, 1, 64, 64), (140, 31, 2, 64, 16)])
def test_attention_of_any_mask(S, n, old, G, D, page):
    """Masks that are no trees: rows that see nothing new (or nothing at all), tokens after them, not themselves."""
    r = random.Random(n)
    pr = problem([n - 1, n - 1], [old, 0], 2 * G, 2, D, page, BF, seed=n)
    rows = []
    for i in range(2 * n):
        kind = r.randrange(4)
        rows.append([] if kind == 0 else [j for j in range(n) if r.random() < (0.02, 0.5, 0.9)[kind - 1]])
    got = check_attention(S, pr, rows, words=(n + 31) // 32 + 2)
    empty = [t for t in range(n, 2 * n) if not rows[t]]
    assert empty and (got["lse"][empty] == -math.inf).all() and (got["out"][empty] == 0).all()


def test_attention_of_causal_masks_is_chunk_attention(S):
    from constrained_logits_sampling_gb300.speculative import ChunkAttention
    for n, G in ((4, 4), (30, 4), (70, 2), (200, 2)):
        pr = problem([n - 1] * 3, [100, 0, 1500], 2 * G, 2, 64, 16, BF, seed=n)
        args = tensors(pr)
        rows = [list(range(i + 1)) for i in range(n)] * 3
        got = S.TreeAttention()(*args, mask=TR.words_of(rows, (n + 31) // 32).cuda(), max_new=n, lse=True)
        want = ChunkAttention()(*args, max_new=n, lse=True)
        # each is off by a rounding of the weights and one of the result, 2^-8 of |v| < 6, and lse by
        # 2^-24 (16 + 8 64) + 2^-22 10 for scores below 64
        assert (got["out"].float() - want["out"].float()).abs().max() <= 2 * 2 * 2.0 ** -8 * 6
        assert (got["lse"] - want["lse"]).abs().max() <= 1e-4


@pytest.mark.parametrize("n,G,page", [(4, 3, 16), (40, 2, 16), (40, 2, 24), (150, 2, 64), (150, 1, 12)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_attention_slots_that_no_row_sees(S, n, G, page, value):
    """New tokens that nobody sees, slots past the length and, with a window, old ones may hold anything."""
    window = 30
    pr = problem([n - 1, n - 1], [90, 200], 2 * G, 2, 64, page, BF, seed=n)
    hidden = {1, n // 2, n - 2}
    _, lines, depth = trees_of([n - 1, n - 1], n, window)
    rows = [[j for j in r if j not in hidden] for r in lines]
    pos = [o + d for o, t in zip((90, 200), depth) for d in t]
    ref = TR.attention(pr, rows, pos, window)
    for b, old in enumerate((90, 200)):
        for x in [old + j for j in hidden] + list(range(old - window + 1)):
            p = int(pr.table[b, x // page])
            pr.k_cache[p, x % page] = pr.v_cache[p, x % page] = value
    check_attention(S, pr, rows, pos, window, ref=ref)


def test_attention_scale_large_scores_and_bounds(S):
    pr = problem([2, 30], [87, 160], 4, 2, 64, 16, FP, seed=5)
    _, rows, _ = trees_of([2, 30], 5)
    check_attention(S, pr, rows, scale=3.0)
    # bits of tokens that are not there are not looked at
    q = tensors(pr)
    mask = TR.words_of(rows, 3)
    full = mask.clone()
    for t in range(pr.T):
        n = 3 if t < 3 else 31
        for j in range(n, 96):
            full[t, j >> 5] |= int(np.uint32(1 << (j & 31)).astype(np.int32))
    a = S.TreeAttention()(*q, mask=mask.cuda(), max_new=31)["out"]
    assert torch.equal(a, S.TreeAttention()(*q, mask=full.cuda(), max_new=31)["out"])
    assert torch.equal(a, S.TreeAttention()(*q, mask=full.cuda()[:, :1])["out"])  # a strided mask, the bound its width


def test_attention_same_bits_streams_and_graphs(S):
    att = S.TreeAttention()
    drafted, old = [40, 3], [700, 900]
    pr = problem(drafted, old, 8, 2, 128, 16, BF, seed=9)
    _, rows, _ = trees_of(drafted, 9)
    first = check_attention(S, pr, rows, handle=att)
    small = problem([0], [30], 8, 2, 128, 16, BF, seed=4)
    for _ in range(3):
        check_attention(S, small, [[0]], handle=att)
        assert torch.equal(check_attention(S, pr, rows, handle=att)["out"], first["out"])
    args = tensors(pr)
    mask = TR.words_of(rows, 2).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = att(*args, mask=mask, max_new=41, stream=side)
    side.synchronize()
    assert torch.equal(got["out"], first["out"])
    out = torch.empty_like(args[0])
    a = att.make_args(*args, mask=mask, max_new=41, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att.apply(a)
    out.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first["out"])


@pytest.mark.parametrize("n,page", [(2, 16), (50, 16), (50, 12)])
def test_attention_bad_sequences(S, n, page):
    """A sequence that cannot be is INVALID and the others are what they were."""
    def make():
        return R.Problem([n] * 5, [80, 200, 150, 90, 64], 4, 2, 64, page, BF, seed=11)

    _, rows, _ = trees_of([n - 1] * 5, 4)
    words = (n + 31) // 32
    mask = TR.words_of(rows, words).cuda()
    pr = make()
    ref, lse, tol, _ = TR.attention(pr, rows)
    pr.table[1, 3] = pr.pages  # a page past the cache
    pr.table[4, 0] = -1
    pr.kv_lens[2] = n - 1  # shorter than its new tokens
    got = S.TreeAttention()(*tensors(pr), mask=mask, max_new=n, lse=True)
    assert got["status"].cpu().tolist() == [0, 2, 2, 0, 2]
    out = got["out"].cpu().double()
    for b in (0, 3):
        assert ((out - ref).abs() <= tol)[b * n:b * n + n].all()
    assert (out[2 * n:3 * n] == 0).all() and (got["lse"][2 * n:3 * n] == -math.inf).all()
    assert torch.isfinite(out).all()  # keys on the bad pages are left out

    pr = make()
    pos = [m - n + min(i, 1) for m in pr.lens for i in range(n)]
    pos[0], pos[2 * n - 1] = 80 - n - 1, 200  # before the tree, and behind it
    got = S.TreeAttention()(*tensors(pr), mask=mask, positions=i32(pos), window=40, max_new=n)
    assert got["status"].cpu().tolist() == [2, 2, 0, 0, 0] and torch.isfinite(got["out"].float()).all()
    pr = make()
    got = S.TreeAttention()(*tensors(pr), mask=mask, max_new=n - 1)
    assert got["status"].cpu().tolist() == [2] * 5 and (got["out"] == 0).all()
    pr.cu = torch.tensor([0, n, 3 * n, 2 * n, 4 * n, 9 * n], dtype=I32)  # back, and past the end
    out = torch.full(pr.q.shape, 5.0, dtype=BF, device="cuda")
    got = S.TreeAttention()(*tensors(pr), mask=torch.zeros(5 * n, 2 * words, dtype=I32, device="cuda"), out=out)
    assert got["status"].cpu().tolist() == [0, 0, 2, 0 if 2 * n <= 90 else 2, 2]
    assert (out[4 * n:] == 5.0).all()  # no sequence owns these rows


def test_attention_far_offsets(S):
    """A cache whose last pages lie past 2^31 elements, and masks whose rows do."""
    page, Hkv, D = 128, 128, 64
    pages = (1 << 31) // (page * Hkv * D) + 4
    k = torch.zeros(pages, page, Hkv, D, dtype=BF, device="cuda")
    v = torch.zeros(pages, page, Hkv, D, dtype=BF, device="cuda")
    for n in (2, 24):
        pr = problem([n - 1], [200 - n], Hkv, Hkv, D, page, BF, seed=12)
        for i, far in enumerate((pages - 1, pages - 2)):
            k[far], v[far] = pr.k_cache[int(pr.table[0, i])].cuda(), pr.v_cache[int(pr.table[0, i])].cuda()
        _, rows, _ = trees_of([n - 1], 2)
        wide = torch.zeros(n, (1 << 31) // (n - 1) + 8, dtype=I32, device="cuda") if n == 2 else None
        mask = TR.words_of(rows, 1).cuda()
        if wide is not None:
            wide[:, :1] = mask
            mask = wide[:, :1]
            assert mask.stride(0) >= 1 << 31
        got = S.TreeAttention()(pr.q.cuda(), k, v, i32([[pages - 1, pages - 2]]), pr.cu.cuda(), pr.kv_lens.cuda(), mask=mask,
                                max_new=n)
        ref, _, tol, _ = TR.attention(pr, rows)
        assert ((got["out"].cpu().double() - ref).abs() <= tol).all()
        del wide, mask


def test_attention_refusals(S):
    pr = problem([3], [36], 4, 2, 64, 16, BF, seed=13)
    _, rows, _ = trees_of([3], 1)
    base, mask = tensors(pr), TR.words_of(rows, 1).cuda()
    att = S.TreeAttention()
    att(*base, mask=mask)
    for kw in (dict(mask=mask[:-1]), dict(mask=mask.float()), dict(mask=mask.cpu()), dict(mask=mask, max_new=33),
               dict(mask=mask, positions=i32([0])), dict(mask=mask.long()), dict(mask=mask[:, 0]),
               dict(mask=mask, window=1 << 31)):
        with pytest.raises(ValueError):
            att(*base, **kw)
    with pytest.raises(Exception) as e:
        att(*base, mask=mask, window=-1)
    assert e.value.code == -9


# ----------------------------------------------------------------------------- append by position

@pytest.mark.parametrize("D,rot,inter", [(128, 128, False), (64, 32, True), (80, 40, False), (33, 10, True)])
def test_append_by_positions(S, D, rot, inter):
    """Each token goes to the slot of its row, rotated by its position."""
    import test_gpu_speculative as G
    pr = R.Problem([9], [60], 4, 2, D, 16, BF, seed=D)
    depth = [0, 1, 1, 2, 2, 2, 3, 1, 4]
    cs, (qw, kw) = G.tables(pr, rot)
    by_slot = cs.clone()
    for i, d in enumerate(depth):
        by_slot[51 + i] = cs[51 + d]
    want_q, q_tol, want_k, k_tol, where = R.append(pr, by_slot, rot, inter, qw, kw)
    q, k, v = (x.contiguous().cuda() for x in (pr.q, pr.k, pr.v))
    kc, vc = gpu(pr.k_cache), gpu(pr.v_cache)
    got = S.KVAppend()(q, k, v, kc, vc, gpu(pr.table), gpu(pr.cu), gpu(pr.kv_lens), cos_sin=gpu(cs), interleaved=inter,
                       q_weight=gpu(qw), k_weight=gpu(kw), positions=i32([51 + d for d in depth]))
    assert got["status"].tolist() == [0]
    assert ((got["q"].cpu().double() - want_q).abs() <= q_tol).all()
    for t, (p, s) in enumerate(where):
        assert ((kc[p, s].cpu().double() - want_k[t]).abs() <= k_tol[t]).all()
        assert torch.equal(vc[p, s].cpu(), pr.v[t])


def test_append_bad_positions(S):
    pr = R.Problem([2, 2, 2], [20, 30, 25], 4, 2, 64, 16, BF, seed=2)
    q, k, v = (x.contiguous().cuda() for x in (pr.q, pr.k, pr.v))
    kc, vc = gpu(pr.k_cache), gpu(pr.v_cache)
    before = kc.clone()
    cs = torch.rand(29, 64).cuda()  # shorter than the second sequence: its slots count for nothing here
    args = (q, k, v, kc, vc, gpu(pr.table), gpu(pr.cu), gpu(pr.kv_lens))
    got = S.KVAppend()(*args, cos_sin=cs, positions=i32([18, -1, 28, 28, 3, 29]))
    assert got["status"].tolist() == [2, 0, 2]
    for t, ok in enumerate([1, 0, 1, 1, 1, 0]):
        b, x = t // 2, pr.lens[t // 2] - 2 + t % 2
        p, s = int(pr.table[b, x // 16]), x % 16
        assert ok == (not torch.equal(kc[p, s].view(torch.int16), before[p, s].view(torch.int16)))
        assert bool(got["q"][t].any()) == bool(ok)
    with pytest.raises(ValueError):
        S.KVAppend()(*args, cos_sin=cs, positions=i32([1]))


# ----------------------------------------------------------------------------- verify

def softmax_rows(rng, n, V, sharp):
    z = rng.standard_normal((n, V)) * sharp
    e = np.exp(z - z.max(1, keepdims=True))
    return (e / e.sum(1, keepdims=True)).astype(np.float32)


def to_type(p, dtype):
    return torch.from_numpy(p).to(dtype)


def batch(sizes, V, seed, draft, dtype=torch.float32, noise=0.5, deep=6, trees=None):
    """A batch as numpy arrays: target, draft rows (one a continued token), ids, parents, offsets, numbers."""
    r, rng = random.Random(seed), np.random.default_rng(seed)
    trees = trees or [TR.tree(r, n, deep, 2 + n // 3) for n in sizes]
    cu = np.concatenate([[0], np.cumsum([len(t) for t in trees])]).astype(np.int32)
    B, N = len(trees), int(cu[-1])
    z = rng.standard_normal((N + B, V)) * 1.5
    soft = lambda a: np.exp(a - a.max(1, keepdims=True)) / np.exp(a - a.max(1, keepdims=True)).sum(1, keepdims=True)  # noqa: E731
    target = to_type(soft(z).astype(np.float32), dtype).float().numpy()
    own = [int(cu[b]) + b + p + 1 for b, t in enumerate(trees) for p in t]
    wanted = sorted(set(own))
    q = soft(z[wanted] + noise * rng.standard_normal((len(wanted), V))).astype(np.float32) if wanted else np.zeros((0, V), np.float32)
    q = to_type(q, dtype).float().numpy()
    rows = np.array([wanted.index(o) for o in own], np.int32)
    x = np.zeros(N, np.int32)
    count = {}
    for i in range(N):
        if draft:
            w = q[rows[i]].astype(np.float64)
            x[i] = rng.choice(V, p=w / w.sum())
        else:
            k = count.get(rows[i], 0)
            count[rows[i]] = k + 1
            x[i] = np.argsort(-q[rows[i]])[min(k, V - 1)]
    u, ul = rng.random(N, np.float32), rng.random(B, np.float32)
    parents = np.array([p for t in trees for p in t], np.int32)
    return dict(target=target, draft=q if draft else None, rows=rows if draft else None, x=x, parents=parents, cu=cu, u=u,
                ul=ul, most=max(len(t) for t in trees))


def run_verify(S, d, dtype=torch.float32, pad=0, max_path=None, draft_rows=True):
    def rows(p):
        if p is None:
            return None
        t = torch.zeros(p.shape[0], p.shape[1] + pad, dtype=dtype, device="cuda")
        t[:, pad // 2:pad // 2 + p.shape[1]] = torch.from_numpy(p).to(dtype).cuda()
        return t[:, pad // 2:pad // 2 + p.shape[1]]

    g = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    got = S.TreeVerifier()(rows(d["target"]), g(d["x"]), g(d["parents"]), g(d["cu"]), g(d["u"]), g(d["ul"]),
                           max_draft=d["most"], max_path=max_path, draft_probs=rows(d["draft"]),
                           draft_rows=g(d["rows"]) if d["draft"] is not None and draft_rows else None)
    return {k: v.cpu().numpy() for k, v in got.items()}


def check_verify(S, d, max_path=None, **kw):
    got = run_verify(S, d, max_path=max_path, **kw)
    most = d["most"] if max_path is None else max_path
    tokens, path, accepted = TR.verify_tree(d["target"], d["draft"], d["rows"], d["x"], d["parents"], d["cu"], d["u"],
                                            d["ul"], most)
    assert (got["status"] == 0).all()
    assert np.array_equal(got["accepted"], accepted)
    assert np.array_equal(got["path"], path)
    assert np.array_equal(got["tokens"], tokens)
    return got


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("sizes,V,dtype,pad,noise", [
    ([0], 7, torch.float32, 0, 0.5), ([1], 33, torch.float32, 0, 0.5), ([7], 100, torch.float32, 6, 1.0),
    ([12, 0, 3, 31, 1], 257, torch.float32, 0, 0.7), ([12, 5, 31, 8], 257, torch.bfloat16, 3, 0.7),
    ([20] * 12, 64, torch.float32, 2, 1.5), ([20] * 12, 1000, torch.bfloat16, 0, 0.3), ([5] * 80, 50, torch.float32, 0, 1.0),
    ([9] * 30, 4, torch.float32, 0, 2.0), ([63, 64, 65], 300, torch.bfloat16, 5, 2.0)])
def test_verify(S, draft, sizes, V, dtype, pad, noise):
    d = batch(sizes, V, len(sizes) + V, draft, dtype, noise)
    check_verify(S, d, dtype=dtype, pad=pad)


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B", [200, 400])  # clusters of two and of four
def test_verify_many(S, draft, B):
    d = batch([6] * B, 40, B, draft, noise=1.0, deep=3)
    got = check_verify(S, d)
    assert got["accepted"].max() >= 2 and got["accepted"].min() == 0


@pytest.mark.parametrize("draft", [True, False])
def test_verify_stars_and_large_trees(S, draft):
    """Many children of one token, most of them refused; and the largest tree."""
    r = random.Random(1)
    d = batch(None, 200, 3, draft, noise=2.0, trees=[[-1] * 60, [-1] * 30 + [3] * 30 + [40] * 30, TR.tree(r, 1023, 30, 40)])
    d["u"][::2] = 0.999  # long runs of refusals
    check_verify(S, d)


@pytest.mark.parametrize("draft", [True, False])
def test_verify_short_paths(S, draft):
    d = batch([20] * 16, 60, 5, draft, noise=0.2)
    full = check_verify(S, d)["accepted"]
    assert full.max() > (3 if draft else 1)  # deep enough for a limit to matter
    for most in (0, 1, 3):
        got = check_verify(S, d, max_path=most)
        assert np.array_equal(got["accepted"], np.minimum(full, most))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("certain", [False, True])
def test_verify_chains_as_the_chain_verifier(S, dtype, certain):
    """Trees without branches: the bits of DraftVerifier."""
    d = batch(None, 5003, 8, not certain, dtype, 0.6, trees=[TR.chain(n) for n in (3, 0, 7, 1, 5, 2)])
    d["rows"] = np.arange(len(d["x"]), dtype=np.int32)
    got = run_verify(S, d, dtype, draft_rows=False)
    g = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    want = S.DraftVerifier()(g(d["target"]).to(dtype), g(d["x"]), g(d["cu"]), g(d["u"]), g(d["ul"]), max_draft=7,
                             draft_probs=None if certain else g(d["draft"]).to(dtype))
    for k in ("tokens", "accepted", "status"):
        assert np.array_equal(got[k], want[k].cpu().numpy()), k


@pytest.mark.parametrize("draft", [True, False])
def test_verify_keeps_the_targets_distribution(S, draft):
    """The first kept token of many requests with three drafted children is distributed as the target's row:
    chi-square over eight tokens, 7 degrees of freedom, below 43 in all but 3 of 10 million draws."""
    rng = np.random.default_rng(17)
    V, B = 8, 60000
    p, q = softmax_rows(rng, 1, V, 1.2)[0], softmax_rows(rng, 1, V, 1.2)[0]
    if draft:
        x = rng.choice(V, size=(B, 3), p=q.astype(np.float64) / q.astype(np.float64).sum())
    else:
        x = np.tile(np.argsort(-q)[:3], (B, 1))
    target = torch.rand(4 * B, V).cuda()  # the children's rows do not matter for the first token
    target /= target.sum(1, keepdim=True)
    target[::4] = torch.from_numpy(p).cuda()
    g = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    got = S.TreeVerifier()(target, g(x.reshape(-1).astype(np.int32)), i32([-1, -1, -1] * B), i32(np.arange(B + 1) * 3),
                           g(rng.random(3 * B, np.float32)), g(rng.random(B, np.float32)), max_draft=3,
                           draft_probs=g(q[None]) if draft else None, draft_rows=i32([0] * (3 * B)) if draft else None)
    assert not got["status"].any()
    seen = torch.bincount(got["tokens"][:, 0].long(), minlength=V).cpu().numpy()
    want = p.astype(np.float64) / p.astype(np.float64).sum() * B
    assert ((seen - want) ** 2 / want).sum() < 43
    rate = (got["accepted"] > 0).float().mean()
    if draft:
        assert rate > 0.3
    else:  # certain children are accepted with their probability: 6 standard deviations of 60000 draws
        assert abs(rate - p[x[0]].sum()) < 6 * 0.5 / B ** 0.5


def test_verify_same_tokens_and_nothing_left(S):
    """Children with the same id; drafts that cover all of the target, so that nothing is left to draw from."""
    V = 6
    p = np.array([[0.5, 0.25, 0.25, 0, 0, 0]] * 5, np.float32)
    for draft in (None, np.array([[0.5, 0.25, 0.25, 0, 0, 0]], np.float32)):
        for u0 in (0.1, 0.9):
            d = dict(target=p, draft=draft, rows=np.zeros(4, np.int32) if draft is not None else None,
                     x=np.array([0, 0, 1, 1], np.int32), parents=np.array([-1, -1, -1, -1], np.int32),
                     cu=np.array([0, 4], np.int32), u=np.array([u0, 0.99999, 0.99999, 0.9], np.float32),
                     ul=np.array([0.7], np.float32), most=4)
            check_verify(S, d)
    d["u"][:] = 1 - 2.0 ** -24  # refused though q = p: u q < p fails for none
    check_verify(S, d)
    d["target"] = np.array([[1, 0, 0, 0, 0, 0]] * 5, np.float32)  # greedy
    d["draft"] = d["rows"] = None
    d["x"][:] = [3, 0, 0, 2]
    got = check_verify(S, d)
    assert got["path"][0, 0] == 1


def test_verify_bad_requests(S):
    d = batch([4] * 9, 30, 2, True, noise=0.3)
    want = run_verify(S, d)
    e = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in d.items()}
    e["parents"][4] = 0           # request 1: not before its child
    e["x"][8] = 30                # 2
    e["u"][12] = 1.0              # 3
    e["ul"][4] = -0.5             # 4
    e["rows"][20] = len(d["draft"])  # 5
    e["target"][6 * 5] = math.nan    # 6: the root's row
    e["parents"][28:32], e["rows"][28:32] = -1, [e["rows"][28], e["rows"][28] + 1, e["rows"][28], e["rows"][28]]  # 7: siblings
    got = run_verify(S, e)
    assert got["status"].tolist() == [0, 2, 2, 2, 2, 2, 2, 2, 0]
    for k in ("tokens", "path", "accepted"):
        assert np.array_equal(got[k][[0, 8]], want[k][[0, 8]])
        assert (got[k][1:8] == (0 if k == "accepted" else -1)).all()
    e = dict(d, most=3)
    assert run_verify(S, e)["status"].tolist() == [2] * 9  # more tokens than the bound
    e = dict(d, cu=np.array([0, 4, 8, 7, 16, 20, 24, 28, 32, 99], np.int32))
    assert run_verify(S, e)["status"].tolist()[2] == 2 and run_verify(S, e)["status"].tolist()[8] == 2


def test_verify_nothing_to_draw_from(S):
    d = batch([2], 20, 2, False)
    d["target"][:] = 0
    got = run_verify(S, d)
    assert got["status"].tolist() == [2] and (got["tokens"] == -1).all()


@pytest.mark.parametrize("V,dtype", [(262144, torch.float32), (262143, torch.bfloat16), (151936, torch.float32)])
@pytest.mark.parametrize("B", [1, 90, 160])  # clusters of eight, four and two
def test_verify_large_vocabularies(S, V, dtype, B):
    """One refusal after another at the largest sizes, against the rule in 64-bit integers on the device."""
    g = torch.Generator(device="cuda").manual_seed(V)
    p = torch.softmax(torch.randn(4, V, device="cuda", generator=g) * 2, 1).to(dtype)
    q = torch.softmax(torch.randn(1, V, device="cuda", generator=g) * 2, 1).to(dtype)
    x = torch.multinomial(q[0].float(), 3, replacement=True, generator=g).to(I32)
    u = torch.full((3,), 1 - 2.0 ** -24, device="cuda")  # refused unless p is far above
    ul = torch.rand(B, device="cuda", generator=g)
    got = S.TreeVerifier()(p.repeat(B, 1), x.repeat(B), i32([-1] * 3 * B), i32(list(range(0, 3 * B + 1, 3))), u.repeat(B), ul,
                           max_draft=3, draft_probs=q, draft_rows=i32([0] * (3 * B)))
    assert not got["status"].any()
    P = (p[0].float() * 2.0 ** 40).long()
    c = s = torch.ones((), device="cuda")
    W, acc = None, None
    for i in range(3):
        y = q[0].float()
        have = p[0, x[i].long()].double() if W is None else W[x[i].long()].double() * 2.0 ** -40
        if float(u[i]) * float(y[x[i].long()] * s) < float(have):
            acc = i
            break
        c = s if W is None else c + s
        W = (P - ((y * c).clamp(max=2.0) * 2.0 ** 40).long()).clamp(min=0)
        s = (W.sum().float() * 2.0 ** -40).clamp(max=1.0)
    if acc is not None:
        assert (got["path"][:, 0] == acc).all()
        W = (p[acc + 1].float() * 2.0 ** 40).long()
    C = W.cumsum(0)
    k31 = (ul * 2.0 ** 31).long()
    k = k31 * (C[-1] >> 31) + ((k31 * (C[-1] & (2 ** 31 - 1))) >> 31)
    want = torch.searchsorted(C, k, right=True).to(I32)
    assert torch.equal(got["tokens"].gather(1, got["accepted"].long()[:, None])[:, 0], want)


def test_verify_streams_graphs_and_refusals(S):
    d = batch([6, 9], 500, 4, True)
    want = run_verify(S, d)
    g = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    args = [g(d[k]) for k in ("target", "x", "parents", "cu", "u", "ul")]
    v = S.TreeVerifier()
    kw = dict(max_draft=9, draft_probs=g(d["draft"]), draft_rows=g(d["rows"]))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = v(*args, **kw, stream=side)
    side.synchronize()
    assert np.array_equal(got["tokens"].cpu().numpy(), want["tokens"])
    wide = torch.full((2, 13), -7, dtype=I32, device="cuda")
    a = v.make_args(*args, **kw, tokens=wide[:, 1:11])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        v.apply(a)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(wide[:, 1:11].cpu().numpy(), want["tokens"])
    assert (wide[:, 0] == -7).all() and (wide[:, 11:] == -7).all()
    with pytest.raises(ValueError):
        v(*args, max_draft=9, draft_probs=g(d["draft"]))  # a row a token, unless told
    with pytest.raises(ValueError):
        v(*args, max_draft=9, draft_rows=g(d["rows"]))
    with pytest.raises(ValueError):
        v(args[0].half(), *args[1:], **kw)
    with pytest.raises(ValueError):
        v(*args[:2], args[2][:-1], *args[3:], **kw)
    with pytest.raises(ValueError):
        v.make_args(*args, **kw, tokens=wide[:, :9])
    with pytest.raises(Exception) as e:
        v(*args, **dict(kw, max_path=10))
    assert e.value.code == -9


# ----------------------------------------------------------------------------- together

def example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tree_step.py")
    spec = importlib.util.spec_from_file_location("tree_step", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


def test_example_step(S):
    """The example's loop: kept tokens are those of the rule on the probabilities that the step used, each
    row's logits are those of its line of tokens run as a chain on a cache of its own, and after the steps
    the cache holds what a plain pass over the kept tokens writes, both within the rounding of the
    activations (bf16)."""
    ex = example()
    B, V, width, depth = 3, 300, 3, 3
    shape = dict(vocab=V, Hq=4, Hkv=2, D=64, max_len=192)
    target, draft = ex.TreeDecoder(layers=2, seed=0, pages=60, **shape), ex.TreeDecoder(layers=1, seed=0, pages=60, **shape)
    loop = ex.TreeLoop(target, draft, B, 192, width, depth)
    prompt = [5 * i % V for i in range(1, 42)]
    loop.prefill(prompt)
    page0 = loop.target.table[0, 0]
    kept = [list(prompt) for _ in range(B)]
    for _ in range(6):
        before = loop.target.lens.clone()
        out = loop.step()
        used = {n: t.cpu().numpy() if torch.is_tensor(t) else t for n, t in loop.used.items()}
        tokens, path, accepted = TR.verify_tree(used["target_probs"], None, None, used["draft_tokens"], used["parents"],
                                                used["cu_draft"], used["u_accept"], used["u_sample"], depth)
        assert np.array_equal(out["tokens"].cpu().numpy(), tokens)
        assert np.array_equal(out["path"].cpu().numpy(), path)
        assert np.array_equal(out["accepted"].cpu().numpy(), accepted)
        assert torch.equal(loop.target.lens[1:].cpu(), before[1:].cpu() + 1 + torch.from_numpy(accepted))
        # every row's probabilities against its own line of tokens, run alone
        x = used["draft_tokens"].reshape(B, -1)
        for b in range(B):
            for i, p in enumerate(used["parents"][:x.shape[1]]):
                line, at = [x[b, i]], p
                while at >= 0:
                    line, at = [x[b, at]] + line, used["parents"][at]
                if i % 4 == 1:
                    want = alone(ex, shape, kept[b] + [int(t) for t in line])
                    got = torch.from_numpy(used["target_probs"][b * (x.shape[1] + 1) + 1 + i]).log() * loop.T
                    want = want - want.logsumexp(0)
                    got = got - got.logsumexp(0)
                    # activations are rounded to bf16 (2^-8) some twenty times along the two layers; such errors
                    # add up like their square root, and a logit is a sum over the row
                    size = want.std()
                    assert ((got - want).abs() <= 2 * 8 * 2.0 ** -8 * 20 ** 0.5 * size).all()
            kept[b] += [int(t) for t in tokens[b, :accepted[b] + 1]]
    assert int(loop.target.pool.refs[int(page0)]) == B + 1  # the prompt's first page is still everybody's
    held = loop.target.held.tolist()
    assert held == [-(-n // 16) for n in loop.target.lens.tolist()]
    used_pages = {int(p) for b in range(B + 1) for p in loop.target.table[b, :held[b]]}
    assert int((loop.target.pool.refs > 0).sum()) == len(used_pages)
    # keys and values of all layers: of the first layer they depend on the token and its position alone
    fresh = ex.TreeDecoder(layers=2, seed=0, pages=60, **shape)
    for b in range(B):
        n = int(loop.target.lens[b + 1])
        assert n == len(kept[b]) - 1
        table = torch.arange(12, dtype=I32, device="cuda")[None]
        fresh(i32(kept[b][:n]), table, i32([0, n]), i32([n]), n)
        row = loop.target.table[b + 1]
        for c, w in ((target.k_cache, fresh.k_cache), (target.v_cache, fresh.v_cache)):
            got = torch.stack([c[0, int(row[j // 16]), j % 16] for j in range(n)]).float()
            want = torch.stack([w[0, j // 16, j % 16] for j in range(n)]).float()
            # one product of bf16 numbers in float32, in other orders, rounded once
            assert (got - want).abs().max() <= 2 * 2.0 ** -8 * want.abs().max()


def alone(ex, shape, tokens):
    """Logits after a line of tokens, by ChunkAttention on a cache of its own."""
    key = tuple(sorted(shape.items()))
    if key not in alone.models:
        alone.models[key] = ex.TreeDecoder(layers=2, seed=0, pages=12, **shape)
    n = len(tokens)
    table = torch.arange(12, dtype=I32, device="cuda")[None]
    return alone.models[key](i32(tokens), table, i32([0, n]), i32([n]), n)[-1].cpu()


alone.models = {}


def test_example_runs(S):
    example().main(steps=2, batch=2, vocab=500)


STALLS = [(1, 0), (1, 1), (2, 0), (3, 0), (4, 0), (5, 1), (6, 0), (6, 1), (7, 0), (8, 0), (8, 2), (9, 0), (9, 3), (10, 0),
          (10, 1), (11, 0), (12, 1), (13, 0), (13, 1)]


@pytest.mark.parametrize("barrier,slot", STALLS)
@pytest.mark.parametrize("D,page,dtype,G,Hkv,B", [(128, 16, BF, 4, 3, 60), (64, 8, FP, 2, 4, 260), (64, 12, BF, 4, 4, 260),
                                                  (128, 24, FP, 8, 3, 40)])
def test_attention_wait_that_runs_out(S, D, page, dtype, G, Hkv, B, barrier, slot):
    """A barrier of the chunk kernel, one by one and in pairs, waits for what never comes, for a
    millisecond: the call ends, its sequences and those of later calls on the handle are OVERFLOW, nothing
    outside its rows is written, and another handle is not affected."""
    import time

    import test_gpu_speculative as G0
    OVERFLOW = 1
    att, fresh = S.TreeAttention(), S.TreeAttention()
    new = [46 if b % 3 else 21 for b in range(B)]
    q, k, v, table, cu, lens = G0.batch(new, [46 + 97 * b % 700 for b in range(B)], G * Hkv, Hkv, D, page, dtype, 2)
    T, guard = sum(new), 200
    mask = torch.full((T, 2), -1, dtype=I32, device="cuda")
    want = fresh(q, k, v, table, cu, lens, mask=mask, max_new=46, lse=True)
    assert not want["status"].any()
    room = torch.full((T + 2 * guard, G * Hkv, D), 3.0, dtype=dtype, device="cuda")
    status = torch.full((B,), -5, dtype=I32, device="cuda")
    args = att.make_args(q, k, v, table, cu, lens, mask=mask, max_new=46, out=room[guard:guard + T], row_status=status)
    assert att._L.clsample_debug_attention_stall(att._h, barrier, slot, 2_000_000) == 0
    torch.cuda.synchronize()
    start = time.time()
    att.apply(args)
    torch.cuda.synchronize()
    assert time.time() - start < 10
    # nobody waits for keys that TMA copies to land, for the end of a CTA's last units, for half of the
    # weights where all are there already, or for a second unit where a CTA has one
    boxes = page % 8 == 0 and 128 % page == 0
    if barrier in (1, 2, 11) or (boxes and barrier in (5, 7)):
        if not status.any():
            assert barrier == 11 or torch.equal(room[guard:guard + T], want["out"])
            return
    assert (status == OVERFLOW).all()
    assert (room[:guard] == 3).all() and (room[guard + T:] == 3).all()
    assert att._L.clsample_debug_attention_stall(att._h, 0, 0, 1) == 0
    later = att(q, k, v, table, cu, lens, mask=mask, max_new=46)
    assert (later["status"] == OVERFLOW).all() and torch.equal(later["out"], want["out"])
    again = fresh(q, k, v, table, cu, lens, mask=mask, max_new=46, lse=True)
    assert not again["status"].any() and torch.equal(again["out"], want["out"])
