"""Checked calls keep what they use: a graph that has captured one needs it for as long as it is replayed."""
import gc
import weakref

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
I32, BF = torch.int32, torch.bfloat16


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from constrained_logits_sampling_gb300 import build, pages, speculative, tree
    build.build()
    return pages, speculative, tree


def graph_of(fn):
    fn()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    return g


def litter():
    """Memory that was freed holds other things."""
    gc.collect()
    torch.cuda.synchronize()
    room = [torch.full((n,), -1, dtype=torch.int64, device="cuda") for n in (1, 2, 8, 32, 64, 128, 512, 4096) for _ in range(20)]
    torch.cuda.synchronize()
    return room


def test_a_pools_call_keeps_the_pool(M):
    pages = M[0]
    n = 64
    table = torch.full((4, 16), -1, dtype=I32, device="cuda")
    held, lens = (torch.zeros(4, dtype=I32, device="cuda") for _ in range(2))
    new = torch.full((4,), 5, dtype=I32, device="cuda")
    copies, free = torch.empty(4, 3, dtype=I32, device="cuda"), torch.empty(1, dtype=I32, device="cuda")

    def capture():
        pool = pages.PagePool(n, 2)
        calls = (pool.reserve_args(table, held, lens, new, copies=copies, free_pages=free),
                 pool.trim_args(table, held, lens))
        return weakref.ref(pool), calls, graph_of(lambda: [pool.apply(c) for c in calls])

    pool, calls, g = capture()
    room = litter()
    assert pool() is not None
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert free.tolist() == [n - 12] and not pool().refs.any() and (held == 0).all()
    assert all((t == -1).all() for t in room)
    del calls, room
    gc.collect()
    assert pool() is None


@pytest.mark.parametrize("by_mask", [False, True])
def test_a_calls_arguments_keep_the_attention_object(M, by_mask):
    kind = M[2].TreeAttention if by_mask else M[1].ChunkAttention
    T, B = 24, 4
    torch.manual_seed(1)
    q = torch.randn(T, 4, 64, device="cuda").to(BF)
    k, v = (torch.randn(40, 16, 1, 64, device="cuda").to(BF) for _ in range(2))
    table = torch.arange(40, dtype=I32, device="cuda").view(B, 10)
    cu = torch.arange(0, T + 1, T // B, dtype=I32, device="cuda")
    lens = torch.full((B,), 155, dtype=I32, device="cuda")
    kw = dict(mask=torch.full((T, 1), -1, dtype=I32, device="cuda")) if by_mask else {}
    out = torch.zeros_like(q)

    def capture():
        att = kind()
        args = att.make_args(q, k, v, table, cu, lens, max_new=T // B, out=out, **kw)
        return weakref.ref(att), args, graph_of(lambda: att.apply(args))

    att, args, g = capture()
    want = out.clone()
    room = litter()
    assert att() is not None
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all((t == -1).all() for t in room)
    del args
    gc.collect()
    assert att() is None
