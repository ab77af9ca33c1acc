"""Waits of the attention kernel that give up: every call ends, and what it says of itself is true."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, FP = torch.bfloat16, torch.float16
I32 = torch.int32


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from constrained_logits_sampling_gb300 import build, tree
    build.build()
    return tree


@pytest.mark.parametrize("cycles", [1, 3000, 20000, 100000])
@pytest.mark.parametrize("by_mask", [False, True])
@pytest.mark.parametrize("D,page,dtype,G,Hkv,B", [(128, 16, BF, 4, 3, 60), (128, 24, FP, 8, 3, 40), (64, 12, BF, 4, 4, 260),
                                                  (64, 8, FP, 2, 4, 260), (128, 48, BF, 8, 2, 7)])
def test_attention_waits_of_any_length(S, D, page, dtype, G, Hkv, B, by_mask, cycles):
    """No barrier stalls, but a wait may give up after few looks, wherever a CTA then is: the call ends, either
    right or with all its sequences OVERFLOW, nothing outside its rows is written, and another handle is not
    affected."""
    import time

    import test_gpu_speculative as G0
    kind = S.TreeAttention if by_mask else S.ChunkAttention
    fresh = kind()
    new = [46 if b % 3 else 21 for b in range(B)]
    q, k, v, table, cu, lens = G0.batch(new, [46 + 97 * b % 700 for b in range(B)], G * Hkv, Hkv, D, page, dtype, 2)
    T, guard = sum(new), 200
    kw = dict(mask=torch.full((T, 2), -1, dtype=I32, device="cuda")) if by_mask else {}
    want = fresh(q, k, v, table, cu, lens, max_new=46, **kw)
    assert not want["status"].any()
    for _ in range(20):
        att = kind()
        room = torch.full((T + 2 * guard, G * Hkv, D), 3.0, dtype=dtype, device="cuda")
        status = torch.full((B,), -5, dtype=I32, device="cuda")
        args = att.make_args(q, k, v, table, cu, lens, max_new=46, out=room[guard:guard + T], row_status=status, **kw)
        assert att._L.clsample_debug_attention_stall(att._h, 1, 255, cycles) == 0  # there is no slot 255
        torch.cuda.synchronize()
        start = time.time()
        att.apply(args)
        torch.cuda.synchronize()
        assert time.time() - start < 10
        assert (status == 1).all() or (not status.any() and torch.equal(room[guard:guard + T], want["out"]))
        assert (room[:guard] == 3).all() and (room[guard + T:] == 3).all()
    again = fresh(q, k, v, table, cu, lens, max_new=46, **kw)
    assert not again["status"].any() and torch.equal(again["out"], want["out"])
