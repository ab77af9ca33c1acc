"""Tree verification on each size of cluster that a number of requests leads to."""
import numpy as np
import pytest

import test_gpu_tree as T
import tree_reference as TR
from test_gpu_tree import S  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
I32 = torch.int32


def requests(ctas):
    """The most requests that are verified by clusters of so many CTAs."""
    slots = 4 * torch.cuda.get_device_properties(0).multi_processor_count
    sizes = {c: slots // c for c in (16, 8, 4)}
    sizes[2] = slots // 4 + 9
    B = sizes[ctas]
    assert next((c for c in (16, 8, 4) if B * c <= slots), 2) == ctas
    return B


@pytest.mark.parametrize("ctas", [16, 8, 4, 2])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
def test_each_cluster(S, ctas, dtype, draft):  # noqa: F811
    """Against exact rationals, with fewer vectors than CTAs and with more."""
    B = requests(ctas)
    for V, pad in ((17, 0), (201, 3)):
        d = T.batch([n % 6 for n in range(B)], V, ctas + V, draft, dtype, noise=1.0, deep=4)
        got = T.check_verify(S, d, dtype=dtype, pad=pad)
        # (a certain child of 201 tokens is accepted in one of about twenty requests, two in a row hardly ever)
        assert got["accepted"].max() >= (2 if draft else 1) and got["accepted"].min() == 0


@pytest.mark.parametrize("ctas", [8, 4, 2])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
def test_each_cluster_as_alone(S, ctas, dtype, draft):  # noqa: F811
    """A large vocabulary: what a request gets does not depend on how many others there are."""
    B, V = requests(ctas), 100003
    trees = [TR.tree(TR.rng(b), 1 + b % 4, 3, 3) for b in range(B)]
    n = [len(t) for t in trees]
    cu = np.concatenate([[0], np.cumsum(n)])
    g = torch.Generator(device="cuda").manual_seed(ctas)
    z = torch.randn(sum(n) + B, V, device="cuda", generator=g) * 2
    p = torch.softmax(z, 1).to(dtype)
    own = torch.tensor([int(cu[b]) + b + x + 1 for b, t in enumerate(trees) for x in t], device="cuda")
    q = torch.softmax(z + torch.randn(z.shape, device="cuda", generator=g), 1).to(dtype)
    x = torch.multinomial(q[own].float(), 1, generator=g)[:, 0].to(I32)
    u, ul = (torch.rand(m, device="cuda", generator=g) for m in (sum(n), B))
    u[::2] = 1 - 2.0 ** -24
    rows = own.to(I32) if draft else None

    def run(first, last):
        a, b = int(cu[first]), int(cu[last])
        m = b - a + last - first
        kw = dict(draft_probs=q, draft_rows=rows[a:b]) if draft else {}
        return S.TreeVerifier()(p[a + first:a + first + m], x[a:b], T.i32([i for t in trees[first:last] for i in t]),
                                T.i32(list(cu[first:last + 1] - a)), u[a:b], ul[first:last], max_draft=4, **kw)

    got = run(0, B)
    assert not got["status"].any() and got["accepted"].min() == 0
    assert got["accepted"].max() >= 1 or not draft  # (a certain child of so many tokens is hardly ever accepted)
    for b in range(0, B, max(1, B // 25)):
        one = run(b, b + 1)
        for k in ("tokens", "path", "accepted", "status"):
            assert torch.equal(got[k][b:b + 1], one[k]), (b, k)
