"""Pages of a cache on the GPU: the pool against plain Python, moves bit for bit (tree_reference)."""
import random

import numpy as np
import pytest

import spec_reference as R
import tree_reference as TR

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, FP, I32 = torch.bfloat16, torch.float16, torch.int32


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from constrained_logits_sampling_gb300 import build, pages
    build.build()
    return pages


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def offsets(n):
    return i32([0] + list(np.cumsum(n)))


# ----------------------------------------------------------------------------- pool

class Both:
    """A pool on the device and one in Python, side by side."""

    def __init__(self, G, pages, page, B, width, extra=0):
        self.pool, self.ref = G.PagePool(pages, page), TR.Pool(pages, page, B, width)
        self.room = torch.full((B, width + extra), -1, dtype=I32, device="cuda")
        self.table = self.room[:, :width]
        self.held, self.lens = torch.zeros(B, dtype=I32, device="cuda"), torch.zeros(B, dtype=I32, device="cuda")

    def state(self):
        return self.table, self.held, self.lens

    def set_lens(self, lens):
        self.ref.lens = list(lens)
        self.lens.copy_(i32(lens))

    def same(self):
        r, n = self.ref, self.pool.num_pages
        assert self.pool.refs.tolist() == r.refs
        assert self.held.tolist() == r.held and self.lens.tolist() == r.lens
        assert self.table.tolist() == r.table
        bits = self.pool.free_bits.cpu().numpy().view(np.uint8)
        assert np.unpackbits(bits, bitorder="little").tolist() == [int(x == 0) for x in r.refs] + [0] * (len(bits) * 8 - n)

    def fork(self, src, dst):
        got = self.pool.fork(*self.state(), i32(src), i32(dst)).tolist()
        assert got == self.ref.fork(src, dst)
        self.same()
        return got

    def reserve(self, new):
        got = self.pool.reserve(*self.state(), i32(new))
        copies, status, free = self.ref.reserve(new)
        assert got["status"].tolist() == status
        assert got["copies"].tolist() == copies and got["free"].tolist() == [free]
        self.same()
        return status

    def trim(self):
        got = self.pool.trim(*self.state()).tolist()
        assert got == self.ref.trim()
        self.same()
        return got


@pytest.mark.parametrize("pages,page,B,width,seed", [(40, 4, 6, 12, 1), (33, 1, 5, 30, 2), (400, 16, 20, 25, 3), (65, 3, 9, 20, 4),
                                                     (3000, 8, 100, 40, 5), (31, 5, 3, 15, 6)])
def test_pool_against_python(G, pages, page, B, width, seed):
    """Random lives: sequences grow, fork, are cut back over what they share, and end."""
    r, both = random.Random(seed), Both(G, pages, page, B, width, extra=seed % 3)
    seen = set()
    for _ in range(60):
        kind = r.randrange(5)
        lens = list(both.ref.lens)
        if kind <= 1:
            new = [r.choice([0, 0, 1, 1, 3, page, r.randint(0, 3 * page)]) for _ in range(B)]
            status = both.reserve(new)
            seen.update(status)
            if not any(status):
                both.set_lens([m + n for m, n in zip(lens, new)])
        elif kind == 2:
            k = r.randint(1, max(1, B // 3))
            seen.update(both.fork([r.randrange(B) for _ in range(k)], [r.randrange(B) for _ in range(k)]))
        elif kind == 3:  # back to less, without giving pages back yet
            both.set_lens([r.choice([m, m, max(0, m - r.randint(0, 2 * page))]) for m in lens])
        else:
            both.set_lens([m if r.random() < 0.6 else 0 for m in lens])
            both.trim()
    assert 0 in seen and len(seen) > 1
    both.set_lens([0] * B)
    assert both.trim() == [0] * B and both.ref.refs == [0] * pages


def test_pool_the_last_writer_keeps_a_shared_page(G):
    both = Both(G, 20, 4, 4, 4)
    both.reserve([6, 0, 0, 0])
    both.set_lens([6, 0, 0, 0])
    both.fork([0, 0, 0], [1, 2, 3])
    page = both.ref.table[0][1]
    both.reserve([1, 1, 1, 1])
    assert [row[1] == page for row in both.ref.table] == [False, False, False, True]
    both.set_lens([7] * 4)
    both.reserve([1, 0, 0, 1])  # nothing is shared any more where they write
    assert both.ref.refs[both.ref.table[0][0]] == 4


def test_pool_not_enough_pages(G):
    """Nothing happens, every sequence that needs a page is told, and the next call works."""
    both = Both(G, 8, 4, 4, 10)
    both.reserve([10, 3, 0, 0])
    both.set_lens([10, 3, 0, 0])
    both.fork([0], [2])
    assert both.reserve([3, 1, 3, 8]) == [1, 0, 1, 1]
    assert both.reserve([3, 1, 3, 0]) == [0, 0, 0, 0]
    assert both.reserve([0, 0, 0, 1]) == [0, 0, 0, 0]
    assert both.ref.refs.count(0) == 0


def test_pool_many_sequences_and_long_rows(G):
    """More sequences than a block has threads, prompts of many pages, a pool of more than 2^20 pages."""
    B = 2500
    both = Both(G, 40000, 2, B, 30)
    r = random.Random(2)
    new = [r.randint(0, 9) for _ in range(B)]
    both.reserve(new)
    both.set_lens(new)
    src = [b for b in range(0, B, 5)]
    both.set_lens([m if b % 5 != 1 else 0 for b, m in enumerate(both.ref.lens)])
    both.trim()
    both.fork(src, [b + 1 for b in src])
    both.reserve([r.randint(0, 40) for _ in range(B)])
    both.trim()
    big = G.PagePool((1 << 20) + 77, 16)
    table = torch.full((3, 9000), -1, dtype=I32, device="cuda")
    held, lens = torch.zeros(3, dtype=I32, device="cuda"), torch.zeros(3, dtype=I32, device="cuda")
    got = big.reserve(table, held, lens, i32([9000 * 16, 1, 5000 * 16]))
    assert got["status"].tolist() == [0, 0, 0] and got["free"].tolist() == [(1 << 20) + 77 - 14001]
    assert torch.equal(table[0], torch.arange(9000, dtype=I32, device="cuda")) and table[1, 0] == 9000
    assert torch.equal(table[2, :5000], torch.arange(9001, 14001, dtype=I32, device="cuda"))
    lens.copy_(i32([0, 1, 40000]))
    assert big.trim(table, held, lens).tolist() == [0, 0, 0]
    assert int(big.refs.sum()) == 1 + 2500 and held.tolist() == [0, 1, 2500]
    refs = big.refs.clone()
    refs[:] = 1
    refs[-3:] = 0
    big.load(refs)
    lens.copy_(i32([0, 1, 40000]))
    assert big.reserve(table, held, lens, i32([40, 0, 0]))["status"].tolist() == [0, 0, 0]
    assert table[0, :3].tolist() == [(1 << 20) + 74, (1 << 20) + 75, (1 << 20) + 76]


def test_pool_bad_calls(G):
    both = Both(G, 30, 4, 6, 5)
    both.reserve([9, 5, 20, 1, 0, 0])
    both.set_lens([9, 5, 20, 1, 0, 0])
    assert both.reserve([-1, 16, 1, 0, 21, 20]) == [2, 2, 2, 0, 2, 0]  # 5 + 16 and 21 are past the table
    both.set_lens([-1, 5, 20, 9, 0, 0])
    assert both.reserve([1, 1, 0, 1, 0, 0]) == [2, 0, 0, 2, 0, 0]  # 9 tokens in one page
    assert both.trim() == [2, 0, 0, 2, 0, 0]
    both.set_lens([9, 5, 20, 1, 0, 0])
    both.ref.held[4] = both.ref.held[5] = 9
    both.held[4:] = 9
    assert both.reserve([0, 0, 0, 0, 1, 0]) == [0, 0, 0, 0, 2, 2]
    assert both.trim() == [0, 0, 0, 0, 2, 2]
    both.ref.held[4] = both.ref.held[5] = 0
    both.held[4:] = 0
    assert both.fork([0, 0, 1, 6, 4, -1], [4, 4, 5, 5, 6, 3]) == [2] * 6  # the same dst twice; not there
    assert both.fork([0, 4], [4, 5]) == [2, 0]  # a dst that is a src: the other is a fork of nothing
    assert both.fork([0, 1], [0, 2]) == [2, 2]  # itself; one that holds pages
    for bad in (30, -5, 29):  # not there, or held by nobody
        both.ref.table[0][2] = bad
        both.table[0, 2] = bad
        assert both.fork([0], [4]) == [2]
        assert both.reserve([1, 0, 0, 0, 0, 0]) == [2, 0, 0, 0, 0, 0]
    both.set_lens([1, 5, 20, 1, 0, 0])
    assert both.trim() == [2, 0, 0, 0, 0, 0]


def test_pool_streams_graphs_and_refusals(G):
    both = Both(G, 50, 4, 4, 6)
    copies, status, free = i32([[0] * 3] * 4), i32([0] * 4), i32([0])
    new = i32([3, 0, 0, 1])
    call = both.pool.reserve_args(*both.state(), new, copies=copies, row_status=status, free_pages=free)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both.pool.apply(call)
    for lens in ([0, 0, 0, 0], [3, 0, 0, 1], [6, 0, 0, 2]):  # each replay a call of its own
        both.set_lens(lens)
        graph.replay()
        torch.cuda.synchronize()
        want = both.ref.reserve([3, 0, 0, 1])
        assert (copies.tolist(), status.tolist(), free.tolist()) == (want[0], want[1], [want[2]])
        both.same()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert both.pool.fork(*both.state(), i32([0]), i32([1]), stream=side).shape == (1,)
    torch.cuda.synchronize()
    both.ref.fork([0], [1])
    both.same()
    t, h, n = both.state()
    for bad in ((t.long(), h, n), (t, h[:-1], n), (t, h, n.cpu()), (t[:-1], h, n), (t[:, 0], h, n)):
        with pytest.raises(ValueError):
            both.pool.trim(*bad)
    with pytest.raises(ValueError):
        both.pool.fork(t, h, n, i32([0]), i32([1, 2]))
    with pytest.raises(ValueError):
        both.pool.reserve_args(t, h, n, new, copies=copies[:3])
    with pytest.raises(ValueError):
        both.pool.load(torch.zeros(49, dtype=I32, device="cuda"))
    with pytest.raises(ValueError):
        G.PagePool(-1, 4)
    empty = G.PagePool(0, 4)
    assert empty.reserve(t, i32([0] * 4), i32([0] * 4), i32([0, 1, 0, 0]))["status"].tolist() == [0, 1, 0, 0]


# ----------------------------------------------------------------------------- moves

def cache(layers, pages, page, Hkv, D, dtype, layout, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (pages, page, Hkv, D) if layout == "nhd" else (pages, Hkv, page, D)
    if layers:
        shape = (layers,) + shape
    out = []
    for _ in range(2):
        c = torch.randn(shape, device="cuda", generator=g).to(dtype)
        out.append(c if layout == "nhd" else c.transpose(-3, -2))
    return out


def bits(t):
    return t.contiguous().view(torch.int16)


KEEP = [
    # drafted, old, layers, Hkv, D, page, dtype, layout
    ([63], [700], 1, 8, 128, 16, BF, "nhd"),
    ([5, 0, 31, 12, 1], [0, 3, 100, 15, 16], 3, 2, 64, 16, FP, "nhd"),
    ([20] * 9, [7 * i for i in range(9)], 2, 3, 128, 8, BF, "hnd"),
    ([20, 4], [9, 0], 2, 2, 33, 3, FP, "nhd"),  # pieces of two bytes
    ([20, 4], [9, 0], 0, 2, 20, 5, BF, "hnd"),  # of eight, no dimension of layers
    ([20, 4], [9, 0], 2, 1, 6, 1, BF, "nhd"),  # of four
    ([900], [50], 1, 1, 64, 64, BF, "nhd"),
    ([40] * 300, [i % 50 for i in range(300)], 2, 2, 80, 16, BF, "nhd"),
    ([3], [5], 40, 16, 256, 4, FP, "hnd"),
]


def random_path(r, parents):
    at, path = -1, []
    for i, p in enumerate(parents):
        if p == at and r.random() < 0.7:
            path.append(i)
            at = i
    return path


def pages_for(lens, page, seed):
    need = [(m + page - 1) // page for m in lens]
    order = torch.randperm(sum(need) + 2, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lens), max(need) + 1), -3, dtype=I32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = torch.tensor(order[at:at + m], dtype=I32)
        at += m
    return table, sum(need) + 2


@pytest.mark.parametrize("case", KEEP, ids=lambda c: f"{c[0][:2]}-{c[2]}x{c[3]}x{c[4]}-p{c[5]}-{c[7]}")
def test_keep_path(G, case):
    drafted, old, layers, Hkv, D, page, dtype, layout = case
    r = random.Random(D)
    trees = [TR.tree(r, n, deep=400 if n > 800 else 9, wide=2) for n in drafted]
    paths = [random_path(r, t) for t in trees]
    if len(paths) > 3:
        paths[0], paths[2] = list(range(min(3, drafted[0]))), []  # all in place; nothing accepted
    lens = [o + n + 1 for o, n in zip(old, drafted)]
    table, pages = pages_for(lens, page, D)
    k, v = cache(layers, pages, page, Hkv, D, dtype, layout, D)
    width = max(len(p) for p in paths) + 2
    path = torch.tensor([p + [-1] * (width - len(p)) for p in paths], dtype=I32, device="cuda")
    want = [bits(k).cpu().clone(), bits(v).cpu().clone()]
    for b, p in enumerate(paths):
        for i, x in enumerate(p):
            f, t = old[b] + 1 + x, old[b] + 1 + i
            for w in want:
                w[..., int(table[b, t // page]), t % page, :, :] = w[..., int(table[b, f // page]), f % page, :, :].clone()
    got = G.KeepPath()(k, v, table.cuda(), offsets(drafted), i32(lens), path, i32([len(p) for p in paths]))
    assert got["status"].tolist() == [0] * len(paths)
    assert got["kv_lens"].tolist() == [o + 1 + len(p) for o, p in zip(old, paths)]
    assert torch.equal(bits(k).cpu(), want[0]) and torch.equal(bits(v).cpu(), want[1])


def test_keep_path_bad_requests(G):
    n, lens = [6] * 9, [20] * 9
    table, pages = pages_for(lens, 4, 1)
    path = [[0, 2, 5, -1]] * 9
    acc = [3] * 9
    path[1], path[2], path[3] = [0, 2, 2, -1], [2, 0, 1, -1], [1, 3, 6, -1]  # twice, back, past the tree
    acc[4], acc[5] = 7, -1
    lens[6] = 6           # shorter than its rows
    lens[7] = 25          # longer than its table
    table[8, 4] = pages   # where the last token moves from
    k, v = cache(2, pages, 4, 2, 64, BF, "nhd", 1)
    before = bits(k).clone(), bits(v).clone()
    got = G.KeepPath()(k, v, table.cuda(), offsets(n), i32(lens), i32(path), i32(acc))
    assert got["status"].tolist() == [0] + [2] * 8
    assert got["kv_lens"].tolist() == [20 - 6 + 3] + lens[1:]
    b = table[0].tolist()
    for t, f in ((15, 16), (16, 19)):
        for w in before:
            w[:, b[t // 4], t % 4] = w[:, b[f // 4], f % 4]
    assert torch.equal(bits(k), before[0]) and torch.equal(bits(v), before[1])
    # places where tokens stay are not looked at
    table[0, 3] = -1
    got = G.KeepPath()(k, v, table.cuda(), offsets(n), i32([20] * 9), i32([[0, -1]] * 9), i32([1] * 9))
    assert got["status"].tolist() == [0] * 9
    got = G.KeepPath()(k, v, table.cuda(), i32([0, 6, 3, 9, 15, 21, 27, 33, 39, 45]), i32([20] * 9), i32([[0, -1]] * 9), i32([1] * 9))
    assert got["status"].tolist()[1] == 2


@pytest.mark.parametrize("D", [128, 127])
def test_moves_far_offsets(G, D):
    """Pages and layers past 2^31 elements."""
    page, Hkv = 64, 64
    pages = (1 << 30) // (page * Hkv * D) + 4
    k, v = (torch.zeros(3, pages, page, Hkv, D, dtype=BF, device="cuda") for _ in range(2))
    assert 2 * k.stride(0) > 1 << 31
    table = i32([[pages - 1, 0]])
    rows = torch.randn(3, Hkv, D, device="cuda").to(BF)
    for c in (k, v):
        c[:, pages - 1, 9] = rows
    got = G.KeepPath()(k, v, table, i32([0, 5]), i32([12]), i32([[2]]), i32([1]))
    assert got["kv_lens"].tolist() == [8]
    assert torch.equal(k[:, pages - 1, 7], rows) and torch.equal(v[:, pages - 1, 7], rows)
    assert G.CopyPages()(k, v, i32([[pages - 1, pages - 2, 8]])).tolist() == [0]
    for c in (k, v):
        assert torch.equal(c[:, pages - 2, 7], rows) and not c[:, pages - 2, 8:].any()
        for at in ((pages - 1, 9), (pages - 1, 7), (pages - 2, 7)):
            c[:, at[0], at[1]] = 0
        assert not c.any()


def test_keep_path_of_the_most_columns(G):
    """Columns close to 2^31, where a thread's next one may lie past it."""
    Hkv, D = 4194303, 255
    k, v = (torch.zeros(1, 3, Hkv, D, dtype=BF, device="cuda") for _ in range(2))
    for c, add in ((k, 1), (v, 2)):
        c.view(torch.int16)[0, 2] = (torch.arange(Hkv * D, device="cuda") % 31991 + add).view(Hkv, D).to(torch.int16)
    got = G.KeepPath()(k, v, i32([[0]]), i32([0, 2]), i32([3]), i32([[1]]), i32([1]))
    assert got["status"].tolist() == [0] and got["kv_lens"].tolist() == [2]
    for c in (k, v):
        bits16 = c.view(torch.int16)
        assert torch.equal(bits16[0, 1], bits16[0, 2]) and not bits16[0, 0].any()


@pytest.mark.parametrize("layers,Hkv,D,page,dtype,layout", [
    (3, 2, 128, 16, BF, "nhd"), (2, 3, 64, 7, FP, "hnd"), (0, 2, 33, 5, BF, "nhd"), (2, 1, 20, 64, BF, "hnd"), (1, 5, 6, 3, FP, "nhd"),
    (30, 8, 256, 32, BF, "nhd")])
def test_copy_pages(G, layers, Hkv, D, page, dtype, layout):
    pages = 40
    k, v = cache(layers, pages, page, Hkv, D, dtype, layout, D)
    copies = [[0, 20, page], [1, 21, 1], [1, 22, page // 2], [-1, 5, page], [3, 23, 0], [0, 24, page - 1], [39, 38, page],
              [4, 40, 1], [40, 25, 1], [4, 26, page + 1], [4, 27, -1], [4, -1, 1], [6, 6, page]]
    want = [bits(k).clone(), bits(v).clone()]
    for f, t, n in copies[:7]:
        if f >= 0:
            for w in want:
                w[..., t, :n, :, :] = w[..., f, :n, :, :]
    status = G.CopyPages()(k, v, i32(copies))
    assert status.tolist() == [0] * 7 + [2] * 5 + [0]
    assert torch.equal(bits(k), want[0]) and torch.equal(bits(v), want[1])


def test_moves_streams_graphs_and_refusals(G):
    k, v = cache(2, 6, 4, 2, 64, BF, "nhd", 3)
    copies = i32([[0, 5, 3], [-1, -1, 0]])
    copier, keeper = G.CopyPages(), G.KeepPath()
    graph = torch.cuda.CUDAGraph()
    args = copier.make_args(k, v, copies)
    with torch.cuda.graph(graph):
        copier.apply(args)
    copies[1] = i32([1, 4, 4])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(k[:, 5, :3]), bits(k[:, 0, :3])) and torch.equal(bits(v[:, 4]), bits(v[:, 1]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = (i32([[2, 3]]), i32([0, 2]), i32([4]), i32([[1]]), i32([1]))
    torch.cuda.synchronize()
    got = keeper(k, v, *call, stream=side)
    side.synchronize()
    assert got["kv_lens"].tolist() == [3] and torch.equal(bits(k[:, 2, 2]), bits(k[:, 2, 3]))
    for bad in ((k, v[:, :-1]), (k.float(), v.float()), (k[0], v), (k[0, 0], v[0, 0]), (k.cpu(), v.cpu()),
                (k[:1].expand(2, -1, -1, -1, -1), v)):
        with pytest.raises(ValueError):
            keeper(*bad, *call)
        with pytest.raises(ValueError):
            copier(*bad, copies)
    with pytest.raises(ValueError):
        copier(k, v, copies[:, :2])
    with pytest.raises(ValueError):
        keeper(k, v, call[0], call[1], call[2], call[3][0], call[4])
    lens = i32([4])
    with pytest.raises(Exception) as e:
        keeper.apply(keeper.make_args(k, v, call[0], call[1], lens, call[3], call[4], new_lens=lens))
    assert e.value.code == -9
    wide = cache(1, 4, 4, 2, 257, BF, "nhd", 3)
    with pytest.raises(Exception) as e:
        copier(*wide, copies)
    assert e.value.code == -9


@pytest.mark.parametrize("graph", [False, True])
def test_calls_that_follow_one_another(G, graph):
    """Fork, reserve, copy, a write, a kept path and trim, each of what the one before has left."""
    page, B, pages = 16, 40, 400
    old, n = 500, 6
    pool, keep, copy = G.PagePool(pages, page), G.KeepPath(), G.CopyPages()
    k, v = (torch.randn(3, pages, page, 2, 64, device="cuda").to(BF) for _ in range(2))
    table = torch.full((B, 40), -1, dtype=I32, device="cuda")
    held, lens, more = (torch.zeros(B, dtype=I32, device="cuda") for _ in range(3))
    more[0] = old
    first = pool.reserve(table, held, lens, more)
    lens[0] = old
    assert first["status"].tolist() == [0] * B
    src, dst = i32([0] * (B - 1)), i32(list(range(1, B)))
    new, cu = i32([n + 1] * B), i32([n * b for b in range(B + 1)])
    path, accepted = i32([[1, 3, 5]] * B), i32([b % 4 for b in range(B)])
    copies, after, free = (torch.zeros(s, dtype=I32, device="cuda") for s in ((B, 3), (B,), (1,)))
    status = [torch.full((B,), -1, dtype=I32, device="cuda") for _ in range(5)]
    fork = pool.fork_args(table, held, lens, src, dst, row_status=status[0][1:])
    reserve = pool.reserve_args(table, held, lens, new, copies=copies, row_status=status[1], free_pages=free)
    moved = copy.make_args(k, v, copies, status=status[2])
    kept = keep.make_args(k, v, table, cu, lens, path, accepted, new_lens=after, row_status=status[3])
    trim = pool.trim_args(table, held, lens, row_status=status[4])
    rows = torch.arange(n + 1, device="cuda")
    values = torch.randn(2, 3, B, n + 1, 2, 64, device="cuda").to(BF)
    who = torch.arange(B, device="cuda").view(B, 1)
    start = [t.clone() for t in (table, held, lens, pool.refs, pool.free_bits)]
    before = k[:, table[0, (old - 1) // page].long(), :old % page].clone()

    def work():
        for t, s in zip((table, held, lens, pool.refs, pool.free_bits), start):
            t.copy_(s)
        pool.apply(fork)
        pool.apply(reserve)
        copy.apply(moved)
        at = old + rows
        ids = table[who, (at // page).view(1, -1)].long()
        k[:, ids, at % page], v[:, ids, at % page] = values[0], values[1]
        lens.add_(n + 1)
        keep.apply(kept)
        lens.copy_(after)
        pool.apply(trim)

    def check():
        assert all(s.tolist()[i == 0:] == [0] * (B - (i == 0)) for i, s in enumerate(status))
        assert lens.tolist() == [old + 1 + b % 4 for b in range(B)]
        for b in range(B):
            ids = table[b].tolist()
            last = ids[(old - 1) // page]
            assert torch.equal(k[:, last, :old % page], before)
            for i, j in enumerate([0] + [p + 1 for p in (1, 3, 5)][:b % 4]):
                x = old + i
                assert torch.equal(k[:, ids[x // page], x % page], values[0][:, b, j])
                assert torch.equal(v[:, ids[x // page], x % page], values[1][:, b, j])
        own = (old - 1) // page
        assert len({int(t) for t in table[:, own]}) == B  # written to, so each has its own
        assert held.tolist() == [-(-int(m) // page) for m in lens]

    if graph:
        work()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            work()
        for _ in range(3):
            k[:, table[:, (old - 1) // page].long(), old % page:] = 0
            g.replay()
            torch.cuda.synchronize()
            check()
    else:
        for _ in range(3):
            work()
            torch.cuda.synchronize()
            check()


def test_forked_sequences_attend_as_their_own(G):
    """A prompt forked twice, each child given a token of its own: attention over the shared pages
    equals attention over caches that share nothing, bit for bit."""
    from constrained_logits_sampling_gb300.speculative import ChunkAttention, KVAppend
    g = torch.Generator(device="cuda").manual_seed(1)
    page, Hq, Hkv, D, L = 16, 4, 2, 64, 41
    pool, copier = G.PagePool(20, page), G.CopyPages()
    table = torch.full((3, 6), -1, dtype=I32, device="cuda")
    held, lens = i32([0, 0, 0]), i32([0, 0, 0])
    k, v = cache(1, 20, page, Hkv, D, BF, "nhd", 1)
    assert not pool.reserve(table, held, lens, i32([L, 0, 0]))["status"].any()
    lens[0] = L
    app, att = KVAppend(), ChunkAttention()
    x = torch.randn(L + 3, Hq + 2 * Hkv, D, device="cuda", generator=g).to(BF)
    part = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    prompt, last = x[:L], x[L:]
    app(part(prompt, 0, Hq), part(prompt, Hq, Hq + Hkv), part(prompt, Hq + Hkv, Hq + 2 * Hkv), k[0], v[0], table[:1].contiguous(),
        i32([0, L]), lens[:1].contiguous())
    assert not pool.fork(table, held, lens, i32([0, 0]), i32([1, 2])).any()
    made = pool.reserve(table, held, lens, i32([1, 1, 1]))
    assert not made["status"].any() and made["copies"][2].tolist() == [-1, -1, 0]
    assert not copier(k, v, made["copies"]).any()
    lens += 1
    one = i32([0, 1, 2, 3])
    q = app(part(last, 0, Hq), part(last, Hq, Hq + Hkv), part(last, Hq + Hkv, Hq + 2 * Hkv), k[0], v[0], table, one, lens)["q"]
    got = att(q, k[0], v[0], table, one, lens, max_new=1)
    # the same rows in pages that nobody shares
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    own = torch.arange(9, dtype=I32, device="cuda").view(3, 3)
    for b in range(3):
        rows = torch.cat([prompt, last[b:b + 1]])
        for i in range(L + 1):
            k2[0, int(own[b, i // page]), i % page] = rows[i, Hq:Hq + Hkv]
            v2[0, int(own[b, i // page]), i % page] = rows[i, Hq + Hkv:]
    want = att(q, k2[0], v2[0], own, one, lens, max_new=1)
    assert torch.equal(got["out"], want["out"]) and not got["status"].any()
    lens.zero_()
    assert not pool.trim(table, held, lens).any() and not pool.refs.any()
