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


@pytest.mark.parametrize("B,width,taken", [(4, 1 << 29, 0), (4, 1 << 30, 0), (1030, 1 << 22, 0), (5, 1 << 30, 3)])
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
