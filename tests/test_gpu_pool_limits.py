"""The pool of pages at the ends of its ranges."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
I32 = torch.int32


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from constrained_logits_sampling_gb300 import build, pages
    build.build()
    return pages


@pytest.mark.parametrize("B,width,taken", [(4, 1 << 29, 0), (4, 1 << 30, 0), (1030, 1 << 22, 0), (5, 1 << 30, 3),
                                           (1024, 1 << 20, 0), (1024, (1 << 20) + 1, 0), (2100, 1 << 20, 7)])
def test_sequences_that_lack_more_pages_than_32_bits_count(G, B, width, taken):
    """With pages of one slot sequences may lack up to 2^30 pages each; their sum, 2^31, 2^32 or more, is
    more than the pool has: nothing is done."""
    pages = 70
    pool = G.PagePool(pages, 1)
    table = torch.empty(B, width, dtype=I32, device="cuda")
    held, lens = (torch.zeros(B, dtype=I32, device="cuda") for _ in range(2))
    new = torch.zeros(B, dtype=I32, device="cuda")
    new[0] = taken
    got = pool.reserve(table, held, lens, new)
    assert not got["status"].any() and got["free"].tolist() == [pages - taken] and held[0] == taken
    before = pool.refs.clone()
    new.fill_(width)
    new[0] -= taken
    lens[0] = taken
    got = pool.reserve(table, held, lens, new)
    assert (got["status"] == 1).all() and got["free"].tolist() == [pages - taken]
    assert (got["copies"] == torch.tensor([-1, -1, 0], dtype=I32, device="cuda")).all()
    assert torch.equal(pool.refs, before) and held.tolist() == [taken] + [0] * (B - 1)
    # and the pool still gives out what it has
    new.zero_()
    new[B - 1] = pages - taken
    got = pool.reserve(table, held, lens, new)
    assert not got["status"].any() and got["free"].tolist() == [0] and held[B - 1] == pages - taken
    assert table[B - 1, :pages - taken].tolist() == list(range(taken, pages))


def test_the_call_number_wraps(G):
    """Around the 2^32nd reservation of a pool, where its call number starts anew: of sequences that write to a
    page that they share the last one keeps it, and no page is lost."""
    for start in (-3, -2, -1, 0):
        pool = G.PagePool(12, 4)
        table = torch.full((3, 4), -1, dtype=I32, device="cuda")
        held, lens = (torch.zeros(3, dtype=I32, device="cuda") for _ in range(2))
        i32 = lambda x: torch.tensor(x, dtype=I32, device="cuda")
        # stamps of the calls before, as large as they get
        pool._stamps.fill_(start * (1 << 32) + 3 if start else 0)
        pool._epoch.fill_(start)
        assert not pool.reserve(table, held, lens, i32([6, 0, 0]))["status"].any()
        lens[0] = 6
        for _ in range(3):
            assert not pool.fork(table, held, lens, i32([0, 0]), i32([1, 2])).any()
            shared = int(table[0, 1])
            assert pool.refs[shared] == 3
            got = pool.reserve(table, held, lens, i32([1, 1, 1]))
            assert not got["status"].any()
            assert int(table[2, 1]) == shared and len({int(table[b, 1]) for b in range(3)}) == 3
            assert got["copies"][:2, 0].tolist() == [shared] * 2 and got["copies"][2].tolist() == [-1, -1, 0]
            assert [int(pool.refs[table[b, 1]]) for b in range(3)] == [1, 1, 1]
            assert got["free"].tolist() == [8] and int((pool.refs == 0).sum()) == 8
            lens[1:] = 0
            assert not pool.trim(table, held, lens).any()
            assert int((pool.refs == 0).sum()) == 10


def busy(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)  # some 50 ms


def test_a_new_pool_is_ready_for_any_stream(G):
    """Made while the current stream is busy, in memory that held other things, and used on another stream at
    once."""
    n = 1000
    table = torch.full((1, n), -1, dtype=I32, device="cuda")
    held, lens = (torch.zeros(1, dtype=I32, device="cuda") for _ in range(2))
    new = torch.full((1,), n, dtype=I32, device="cuda")
    side = torch.cuda.Stream()
    for _ in range(3):  # what the pool's arrays are made of
        old = [torch.full((m,), -1, dtype=t, device="cuda") for m, t in ((n, I32), ((n + 31) // 32, I32), (n, torch.int64),
                                                                         (1, I32), (n, I32), (1024, torch.int64))]
    torch.cuda.synchronize()
    del old
    busy(torch.cuda.current_stream())
    pool = G.PagePool(n, 1)
    got = pool.reserve(table, held, lens, new, stream=side)
    torch.cuda.synchronize()
    assert got["status"].tolist() == [0] and got["free"].tolist() == [0]
    assert table[0].tolist() == list(range(n)) and (pool.refs == 1).all()


def test_loaded_counts_on_a_stream(G):
    """load on a stream of its own comes before later calls there, whatever the current stream does."""
    n = 200
    table = torch.full((1, n), -1, dtype=I32, device="cuda")
    held, lens = (torch.zeros(1, dtype=I32, device="cuda") for _ in range(2))
    new = torch.full((1,), n // 2, dtype=I32, device="cuda")
    refs = (torch.arange(n, device="cuda") % 2).to(I32)
    side, pool = torch.cuda.Stream(), G.PagePool(n, 1)
    torch.cuda.synchronize()
    busy(torch.cuda.current_stream())
    pool.load(refs, stream=side)
    got = pool.reserve(table, held, lens, new, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()  # still asleep
    with torch.cuda.stream(side):
        assert got["status"].tolist() == [0] and got["free"].tolist() == [0]
        assert table[0, :n // 2].tolist() == list(range(0, n, 2))


@pytest.mark.parametrize("slots", [(1 << 31) - 1, (1 << 31) - 20000])
def test_copy_of_a_page_of_the_most_slots(G, slots):
    """A page of 2^31 - 1 slots of one element: places past its end are none, though they pass 2^31."""
    page = (1 << 31) - 1
    room = torch.empty(2 * page + 4096, dtype=torch.bfloat16, device="cuda")
    room[2 * page:] = 3.0
    cache = room[:2 * page].view(2, page, 1, 1)
    cache[0].view(torch.int16).random_(-30000, 30000)
    cache[1] = 5.0
    status = G.CopyPages()(cache, cache, torch.tensor([[0, 1, slots]], dtype=I32, device="cuda"))
    assert status.tolist() == [0]
    a, b = (c.view(torch.int16).view(-1) for c in cache)
    assert torch.equal(a[:slots], b[:slots])
    assert (cache[1].view(-1)[slots:] == 5).all() and (room[2 * page:] == 3).all()
