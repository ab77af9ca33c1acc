"""The speculative-step operators on the GPU against 64-bit references (spec_reference)."""
import math

import numpy as np
import pytest

import spec_reference as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from constrained_logits_sampling_gb300 import build, speculative
    build.build()
    return speculative


def gpu(t):
    """On the device with the strides it has here."""
    if t is None:
        return None
    if t.dim() == 4 and not t.is_contiguous():
        return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    return t.cuda()


def fused(pr):
    """q, k, v on the device as slices of one projection."""
    x = torch.cat([pr.q.flatten(1), pr.k.flatten(1), pr.v.flatten(1)], 1).cuda()
    a, b = pr.Hq * pr.D, (pr.Hq + pr.Hkv) * pr.D
    return (x[:, :a].view(pr.T, pr.Hq, pr.D), x[:, a:b].view(pr.T, pr.Hkv, pr.D), x[:, b:].view(pr.T, pr.Hkv, pr.D))


# ----------------------------------------------------------------------------- attention

ATTEND = [
    # new, lens, Hq, Hkv, D, page, dtype, window, layout
    ([1], [1], 4, 4, 64, 16, BF, 0, "nhd"),
    ([1], [777], 32, 8, 128, 16, BF, 0, "nhd"),
    ([1], [5000], 4, 1, 128, 64, FP, 0, "nhd"),
    ([4, 4, 4], [4, 65, 300], 8, 2, 128, 16, BF, 0, "hnd"),
    ([0, 2, 0, 1, 0], [5, 64, 0, 65, 9], 3, 1, 64, 16, FP, 0, "nhd"),
    ([3, 5], [1, 0], 4, 2, 128, 16, BF, 0, "nhd"),  # rows without keys
    ([7, 1], [129, 128], 10, 2, 64, 5, BF, 0, "nhd"),  # pages that end inside a tile, odd group
    ([2, 3], [70, 33], 6, 6, 128, 1, FP, 0, "hnd"),
    ([9], [400], 4, 4, 64, 24, BF, 7, "nhd"),
    ([1, 6], [300, 300], 8, 1, 128, 128, FP, 1, "nhd"),
    ([5, 40], [200, 260], 4, 2, 64, 32, BF, 100, "hnd"),
    ([33], [33], 4, 1, 128, 16, BF, 0, "nhd"),
    ([70, 1, 130], [70, 500, 333], 8, 2, 128, 64, BF, 0, "nhd"),
    ([150], [700], 4, 4, 64, 16, FP, 50, "nhd"),
    ([65, 0, 129], [40, 3, 200], 5, 1, 64, 8, BF, 0, "nhd"),  # chunk longer than its keys
    ([257], [300], 2, 1, 128, 48, FP, 0, "hnd"),
    ([1] * 300, [(7 * i) % 90 for i in range(300)], 2, 1, 64, 16, BF, 0, "nhd"),
    ([6, 7], [450, 200], 8, 2, 128, 16, FP, 0, "nhd"),  # 17 to 32 packed rows
    ([40], [6000], 4, 1, 128, 64, BF, 0, "nhd"),  # a long unit in many parts
    ([30, 2], [2500, 1200], 6, 2, 64, 256, FP, 700, "hnd"),  # pages longer than a tile, a window
    ([100, 20], [2000, 40], 2, 1, 128, 48, BF, 0, "nhd"),  # pages that are no boxes
    ([20 if i % 40 == 0 else 1 for i in range(310)], [25 + (11 * i) % 70 for i in range(310)], 4, 2, 64, 16, BF, 0,
     "nhd"),  # many short sequences beside longer ones
    ([300], [520], 1, 1, 64, 128, BF, 0, "nhd"),  # two row tiles, one head
]


def check_attention(S, pr, window=0, handle=None, **kw):
    att = handle or S.ChunkAttention()
    out = torch.full((pr.T, pr.Hq, pr.D), 7.0, dtype=pr.dtype, device="cuda")
    q = fused(pr)[0]
    args = (q, gpu(pr.k_cache), gpu(pr.v_cache), gpu(pr.table), gpu(pr.cu), gpu(pr.kv_lens))
    got = att(*args, window=window, max_new=max(pr.new), lse=True, out=out, **kw)
    torch.cuda.synchronize()
    ref, lse, tol, lse_tol = R.attention(pr, window, kw.get("scale"))
    err = (got["out"].cpu().double() - ref).abs()
    assert torch.isfinite(got["out"].float()).all()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())
    gl = got["lse"].cpu().double()
    assert torch.equal(gl == -math.inf, lse == -math.inf)
    seen = lse > -math.inf
    assert ((gl - lse)[seen].abs() <= lse_tol[seen]).all()
    assert got["status"].cpu().tolist() == [0] * pr.B
    return got


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"{c[0][:3]}-{c[1][:3]}-{c[2]}x{c[3]}x{c[4]}-p{c[5]}-w{c[7]}")
def test_attention(S, case):
    new, lens, Hq, Hkv, D, page, dtype, window, layout = case
    check_attention(S, R.Problem(new, lens, Hq, Hkv, D, page, dtype, seed=len(lens) + D, layout=layout), window)


@pytest.mark.parametrize("D,page,dtype", [(64, 8, BF), (64, 16, FP), (128, 16, BF), (64, 24, BF)])
def test_attention_units_in_a_row(S, D, page, dtype):
    """CTAs that take several small and large units in a row, whose loads run ahead of the unit
    that is being finished: against a product of all scores in float32 on the device, with the
    bound of R.attention for weights of any distribution (|v| < 6, roundoff of the type)."""
    g = torch.Generator(device="cuda").manual_seed(D + page)
    B, n, Hq, Hkv = 60, 46, 9, 3  # 138 packed rows: a unit of both row tiles
    lens = [n + (37 * b) % 400 for b in range(B)]
    new = [n if b % 3 else 11 for b in range(B)]  # 33 rows: a unit of one
    pages = [(m + page - 1) // page for m in lens]
    table = torch.zeros(B, max(pages), dtype=torch.int32)
    order, at = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(1)).to(torch.int32), 0
    for b, m in enumerate(pages):
        table[b, :m] = order[at:at + m]
        at += m
    table = table.cuda()
    k, v = (torch.randn(sum(pages), page, Hkv, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    q = torch.randn(sum(new), Hq, D, device="cuda", generator=g).to(dtype)
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    att = S.ChunkAttention()
    first = att(q, k, v, table, cu, kv, max_new=n)["out"]
    u, at = R.ROUND[dtype], 0
    for b in range(B):
        m, c = lens[b], new[b]
        ids = table[b, :pages[b]].long()
        kb, vb = (x[ids].reshape(-1, Hkv, D)[:m].double().repeat_interleave(Hq // Hkv, 1) for x in (k, v))
        y = torch.einsum("ihd,jhd->hij", q[at:at + c].double(), kb) / math.sqrt(D)
        hide = torch.arange(m, device="cuda")[None, :] > torch.arange(m - c, m, device="cuda")[:, None]
        w = torch.softmax(y.masked_fill(hide, -math.inf), -1)
        want = torch.einsum("hij,jhd->ihd", w, vb)
        mag = torch.einsum("hij,jhd->ihd", w, vb.abs())
        # as in R.attention: scores are below 64 in size here, so a weight is off by 2^-24 (16 + 8 64) at most
        tol = (u + 2.0 ** -23 * 528) * mag + u * want.abs() + 1e-7 + (m * 6 * 2.0 ** -25 if dtype == FP else 0)
        assert ((first[at:at + c].double() - want).abs() <= tol).all(), b
        at += c
    for _ in range(3):
        assert torch.equal(att(q, k, v, table, cu, kv, max_new=n)["out"], first)


def test_attention_scale_and_large_scores(S):
    """Scores far above the exponent range: the running maximum has to hold them."""
    pr = R.Problem([3, 40], [90, 200], 4, 2, 64, 16, FP, seed=5)
    check_attention(S, pr, scale=3.0)


def test_attention_same_handle_same_bits(S):
    """One handle over calls of different splits leaves its counters ready, and a call's bits
    do not depend on timing."""
    att = S.ChunkAttention()
    pr = R.Problem([1, 2], [3000, 900], 8, 2, 128, 16, BF, seed=3)
    small = R.Problem([1], [30], 8, 2, 128, 16, BF, seed=4)
    chunk = R.Problem([90], [1500], 8, 2, 128, 16, BF, seed=6)
    first = check_attention(S, pr, handle=att)
    for _ in range(3):
        check_attention(S, small, handle=att)
        check_attention(S, chunk, handle=att)
        again = check_attention(S, pr, handle=att)
        assert torch.equal(first["out"], again["out"]) and torch.equal(first["lse"], again["lse"])


def test_attention_other_stream(S):
    pr = R.Problem([4, 1], [700, 900], 8, 2, 64, 16, BF, seed=8)
    att = S.ChunkAttention()
    side = torch.cuda.Stream()
    args = [fused(pr)[0], gpu(pr.k_cache), gpu(pr.v_cache), gpu(pr.table), gpu(pr.cu), gpu(pr.kv_lens)]
    torch.cuda.synchronize()
    got = att(*args, stream=side)
    side.synchronize()
    ref, _, tol, _ = R.attention(pr)
    assert ((got["out"].cpu().double() - ref).abs() <= tol).all()


def test_attention_in_a_graph(S):
    pr = R.Problem([2, 40], [700, 900], 8, 2, 128, 16, BF, seed=9)
    att = S.ChunkAttention()
    q = fused(pr)[0].contiguous()
    out = torch.empty_like(q)
    a = att.make_args(q, gpu(pr.k_cache), gpu(pr.v_cache), gpu(pr.table), gpu(pr.cu), gpu(pr.kv_lens), out=out)
    att.apply(a)
    torch.cuda.synchronize()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att.apply(a)
    out.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("n,page", [(2, 16), (50, 16), (50, 12)])
def test_attention_bad_sequences(S, n, page):
    """A sequence that cannot be is INVALID and the others are what they were."""
    def problem():
        return R.Problem([n] * 5, [80, 200, 150, 90, 64], 4, 2, 64, page, BF, seed=11)

    pr = problem()
    ref, lse, tol, _ = R.attention(pr)
    pr.table[1, 3] = pr.pages  # a page past the cache
    pr.table[4, 0] = -1
    pr.kv_lens[2] = pr.table.shape[1] * page + 1  # longer than its table
    q = fused(pr)[0]
    got = S.ChunkAttention()(q, gpu(pr.k_cache), gpu(pr.v_cache), gpu(pr.table), gpu(pr.cu), gpu(pr.kv_lens), lse=True)
    assert got["status"].cpu().tolist() == [0, 2, 2, 0, 2]
    out = got["out"].cpu().double()
    for b in (0, 3):
        assert ((out - ref).abs() <= tol)[b * n:b * n + n].all()
    assert (out[2 * n:3 * n] == 0).all() and (got["lse"][2 * n:3 * n] == -math.inf).all()
    assert torch.isfinite(out).all()  # keys on the bad pages are left out

    pr = problem()
    pr.kv_lens[0] = -1
    got = S.ChunkAttention()(fused(pr)[0], gpu(pr.k_cache), gpu(pr.v_cache), gpu(pr.table), gpu(pr.cu),
                             gpu(pr.kv_lens))
    assert got["status"].cpu().tolist() == [2, 0, 0, 0, 0]
    pr = problem()
    pr.cu = torch.tensor([0, n, 3 * n, 2 * n, 4 * n, 9 * n], dtype=torch.int32)  # back, and past the end
    out = torch.full(pr.q.shape, 5.0, dtype=BF, device="cuda")
    got = S.ChunkAttention()(fused(pr)[0], gpu(pr.k_cache), gpu(pr.v_cache), gpu(pr.table), gpu(pr.cu),
                             gpu(pr.kv_lens), out=out)
    assert got["status"].cpu().tolist() == [0, 0, 2, 0, 2]
    assert (out[4 * n:] == 5.0).all()  # no sequence owns these rows
    pr = problem()
    got = S.ChunkAttention()(fused(pr)[0], gpu(pr.k_cache), gpu(pr.v_cache), gpu(pr.table), gpu(pr.cu),
                             gpu(pr.kv_lens), max_new=n - 1)
    assert got["status"].cpu().tolist() == [2] * 5 and (got["out"] == 0).all()


def batch(new, lens, Hq, Hkv, D, page, dtype, seed):
    """q, caches, table, offsets and lengths, made on the device."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [(m + page - 1) // page for m in lens]
    order, at = torch.randperm(sum(need), generator=torch.Generator().manual_seed(seed)).to(torch.int32), 0
    table = torch.zeros(len(new), max(need), dtype=torch.int32)
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    k, v = (torch.randn(sum(need), page, Hkv, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    q = torch.randn(sum(new), Hq, D, device="cuda", generator=g).to(dtype)
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    return q, k, v, table.cuda(), cu, torch.tensor(lens, dtype=torch.int32, device="cuda")


STALLS = [(1, 0), (1, 1), (2, 0), (3, 0), (4, 0), (5, 1), (6, 0), (6, 1), (7, 0), (8, 0), (8, 2), (9, 0), (9, 3), (10, 0),
          (10, 1), (11, 0), (12, 1), (13, 0), (13, 1)]


@pytest.mark.parametrize("barrier,slot", STALLS)
@pytest.mark.parametrize("D,page,dtype,Hq", [(128, 16, BF, 9), (64, 8, FP, 6), (64, 12, BF, 9), (128, 24, FP, 6)])
def test_attention_wait_that_runs_out(S, D, page, dtype, Hq, barrier, slot):
    """A barrier of the chunk kernel waits for what never comes, for a millisecond: the call ends,
    all its sequences and those of later calls on the handle are OVERFLOW, nothing outside the
    call's rows is written (the handle's scratch still holds the cuts of a larger call), and another
    handle is not affected."""
    import time
    Hkv, OVERFLOW = 3, 1
    att, fresh = S.ChunkAttention(), S.ChunkAttention()
    big = batch([70] * 90, [70 + 31 * b % 500 for b in range(90)], Hq, Hkv, D, page, dtype, 1)
    want_big = att(*big, max_new=70)
    assert not want_big["status"].any()
    # units of one row tile and of two (with 9 heads); some eight key tiles and two units a CTA
    new = [46 if b % 3 else 11 for b in range(60)]
    small = batch(new, [46 + 97 * b % 1500 for b in range(60)], Hq, Hkv, D, page, dtype, 2)
    want = fresh(*small, max_new=46, lse=True)
    assert not want["status"].any()
    T, guard = sum(new), 300
    room = torch.full((T + 2 * guard, Hq, D), 3.0, dtype=dtype, device="cuda")
    sums = torch.full(((T + 2 * guard) * Hq,), 3.0, device="cuda")
    status = torch.full((60,), -5, dtype=torch.int32, device="cuda")
    args = att.make_args(*small, max_new=46, out=room[guard:guard + T], row_status=status,
                         lse=sums[guard * Hq:(guard + T) * Hq])
    assert att._L.clsample_debug_attention_stall(att._h, barrier, slot, 2_000_000) == 0
    torch.cuda.synchronize()
    start = time.time()
    att.apply(args)
    torch.cuda.synchronize()
    assert time.time() - start < 10
    # nobody waits for keys that TMA copies to land, for the end of a CTA's last units, or for half of
    # the weights where all are there already
    boxes = page % 8 == 0 and 128 % page == 0
    if barrier in (2, 11) or (boxes and barrier == 5):
        if not status.any():
            assert barrier == 11 or torch.equal(room[guard:guard + T], want["out"])
            return
    assert (status == OVERFLOW).all()
    assert (room[:guard] == 3).all() and (room[guard + T:] == 3).all()
    assert (sums[:guard * Hq] == 3).all() and (sums[(guard + T) * Hq:] == 3).all()
    assert att._L.clsample_debug_attention_stall(att._h, 0, 0, 1) == 0
    later = att(*big, max_new=70)
    assert (later["status"] == OVERFLOW).all() and torch.equal(later["out"], want_big["out"])
    again = fresh(*small, max_new=46, lse=True)
    assert not again["status"].any()
    assert torch.equal(again["out"], want["out"]) and torch.equal(again["lse"], want["lse"])


def test_attention_stall_refusals(S):
    att = S.ChunkAttention()
    stall = att._L.clsample_debug_attention_stall
    assert stall(None, 0, 0, 1) == -1
    for bad in ((-1, 0, 1), (14, 0, 1), (1, -1, 1), (1, 256, 1), (1, 0, 0), (1, 0, 4_000_000_001)):
        assert stall(att._h, *bad) == -9


def test_attention_far_offsets(S):
    """A cache whose last pages lie past 2^31 elements."""
    pages, page, Hkv, D = 1050, 128, 128, 128  # 2.2e9 elements, 4.4 GB each
    k = torch.zeros(pages, page, Hkv, D, dtype=BF, device="cuda")
    v = torch.zeros(pages, page, Hkv, D, dtype=BF, device="cuda")
    pr = R.Problem([2], [200], Hkv, Hkv, D, page, BF, seed=12)
    for i, far in enumerate((pages - 1, pages - 2)):
        k[far], v[far] = pr.k_cache[int(pr.table[0, i])].cuda(), pr.v_cache[int(pr.table[0, i])].cuda()
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    got = S.ChunkAttention()(fused(pr)[0], k, v, table, gpu(pr.cu), gpu(pr.kv_lens))
    ref, _, tol, _ = R.attention(pr)
    assert ((got["out"].cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("page", [128, 120])  # copied in boxes, and row by row
def test_attention_far_offsets_of_chunks(S, page):
    """More than 16 packed rows over a cache whose last pages lie past 2^31 elements."""
    Hkv, D = 128, 128
    pages = (1 << 31) // (page * Hkv * D) + 4
    k = torch.zeros(pages, page, Hkv, D, dtype=BF, device="cuda")
    v = torch.zeros(pages, page, Hkv, D, dtype=BF, device="cuda")
    pr = R.Problem([24], [200], Hkv, Hkv, D, page, BF, seed=12)
    for i, far in enumerate((pages - 1, pages - 2)):
        k[far], v[far] = pr.k_cache[int(pr.table[0, i])].cuda(), pr.v_cache[int(pr.table[0, i])].cuda()
    assert (pages - 2) * k.stride(0) > 1 << 31
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    got = S.ChunkAttention()(fused(pr)[0], k, v, table, gpu(pr.cu), gpu(pr.kv_lens))
    ref, _, tol, _ = R.attention(pr)
    assert ((got["out"].cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("n,page", [(3, 16), (30, 16), (30, 12)])
def test_attention_one_sequence_not_finite(S, n, page):
    """Queries that are NaN or infinite, and keys and values of their sequence that are, concern
    nobody else; the slots past each length hold NaN."""
    pr = R.Problem([n] * 5, [90, n, 150, 200, 77], 6, 2, 64, page, BF, seed=17)
    ref, lse, tol, lse_tol = R.attention(pr)
    pr.q[n:2 * n] = math.nan
    pr.q[3 * n:4 * n] = math.inf
    for b, value in ((1, math.inf), (3, math.nan)):
        p = int(pr.table[b, 0])
        pr.k_cache[p, 0] = pr.v_cache[p, 0] = value
    got = S.ChunkAttention()(fused(pr)[0], gpu(pr.k_cache), gpu(pr.v_cache), gpu(pr.table), gpu(pr.cu), gpu(pr.kv_lens),
                             max_new=n, lse=True)
    assert got["status"].cpu().tolist() == [0] * 5
    for b in (0, 2, 4):
        rows = slice(b * n, b * n + n)
        assert ((got["out"].cpu().double() - ref).abs() <= tol)[rows].all()
        assert ((got["lse"].cpu().double() - lse).abs() <= lse_tol)[rows].all()
    assert torch.isnan(got["out"][n:2 * n].float()).all() and torch.isnan(got["out"][3 * n:4 * n].float()).all()


def test_attention_two_handles_at_once(S):
    """Calls of both kernels on two handles and two streams, side by side: the bits of calls alone."""
    shapes = [batch([1 + 3 * (b % 3) for b in range(40)], [300 + 77 * b for b in range(40)], 8, 2, 128, 16, BF, 5),
              batch([70 if b % 5 == 0 else 1 for b in range(400)], [100 + 13 * b % 900 for b in range(400)], 6, 3, 64, 32, FP, 6)]
    most = [7, 70]
    want = [S.ChunkAttention()(*a, max_new=m, lse=True) for a, m in zip(shapes, most)]
    torch.cuda.synchronize()
    handles, streams, got = [S.ChunkAttention() for _ in shapes], [torch.cuda.Stream() for _ in shapes], [[], []]
    for _ in range(20):
        for i, a in enumerate(shapes):
            got[i].append(handles[i](*a, max_new=most[i], lse=True, stream=streams[i]))
    torch.cuda.synchronize()
    for i, calls in enumerate(got):
        for c in calls:
            assert not c["status"].any()
            assert torch.equal(c["out"], want[i]["out"]) and torch.equal(c["lse"], want[i]["lse"])


def test_attention_refusals(S):
    pr = R.Problem([2], [40], 4, 2, 64, 16, BF, seed=13)
    att = S.ChunkAttention()
    q = fused(pr)[0]
    base = [q, gpu(pr.k_cache), gpu(pr.v_cache), gpu(pr.table), gpu(pr.cu), gpu(pr.kv_lens)]

    def call(i=None, t=None, **kw):
        a = list(base)
        if i is not None:
            a[i] = t
        return att(*a, **kw)

    call()
    with pytest.raises(ValueError):
        call(0, q.float())
    with pytest.raises(ValueError):
        call(0, q[:, :, :32])
    with pytest.raises(ValueError):
        call(1, base[1].to(FP))
    with pytest.raises(ValueError):
        call(2, base[2][:-1])
    with pytest.raises(ValueError):
        call(3, base[3].long())
    with pytest.raises(ValueError):
        call(4, base[4][:-1])
    with pytest.raises(ValueError):
        call(4, base[4].cpu())
    with pytest.raises(ValueError):
        call(out=torch.empty(3, 4, 64, dtype=BF, device="cuda"))
    for kw, code in ((dict(window=-1), -9), (dict(scale=0.0), -9), (dict(scale=float("nan")), -9),
                     (dict(max_new=-1), -9)):
        with pytest.raises(Exception) as e:
            call(**kw)
        assert e.value.code == code
    with pytest.raises(Exception) as e:  # 3 query heads on 2 key heads
        call(0, q[:, :3])
    assert e.value.code == -9
    with pytest.raises(Exception) as e:
        wide = torch.zeros(2, 4 * 64 + 1, dtype=BF, device="cuda")
        call(0, wide[:, 1:].view(2, 4, 64))
    assert e.value.code == -10


def test_attention_numbers_past_32_bits(S):
    pr = R.Problem([2], [40], 4, 2, 64, 16, BF, seed=13)
    args = (fused(pr)[0], gpu(pr.k_cache), gpu(pr.v_cache), gpu(pr.table), gpu(pr.cu), gpu(pr.kv_lens))
    att = S.ChunkAttention()
    ref, _, tol, _ = R.attention(pr)
    for kw in (dict(window=(1 << 31) - 1), dict(max_new=(1 << 31) - 1)):  # the bound chooses the kernel
        assert ((att(*args, **kw)["out"].cpu().double() - ref).abs() <= tol).all()
    for kw in (dict(window=(1 << 32) + 5), dict(max_new=(1 << 32) + 1)):
        with pytest.raises(ValueError):
            att(*args, **kw)


@pytest.mark.parametrize("n", [1, 40])
def test_attention_largest_scale(S, n):
    """Scores of zero stay zero up to the largest scale; above it, where the scale in powers of
    two is no longer finite, the call is refused."""
    pr = R.Problem([n], [90], 2, 1, 64, 16, BF, seed=n)
    att = S.ChunkAttention()
    q = torch.zeros_like(fused(pr)[0])
    args = (q, gpu(pr.k_cache), gpu(pr.v_cache), gpu(pr.table), gpu(pr.cu), gpu(pr.kv_lens))
    got = att(*args, max_new=n, scale=2.0e38)["out"]
    assert torch.isfinite(got.float()).all()
    assert torch.equal(got, att(*args, max_new=n, scale=1.0)["out"])
    with pytest.raises(Exception) as e:
        att(*args, max_new=n, scale=2.5e38)
    assert e.value.code == -9


# ----------------------------------------------------------------------------- append

APPEND = [
    # new, lens, Hq, Hkv, D, page, dtype, rot, interleaved, norm, layout
    ([1], [778], 32, 8, 128, 16, BF, 128, False, True, "nhd"),
    ([1], [1], 1, 1, 64, 16, FP, 64, True, False, "nhd"),
    ([4, 4, 4], [4, 70, 300], 8, 2, 128, 64, BF, 128, False, True, "hnd"),
    ([0, 3, 0, 0, 21, 1, 0], [9, 3, 0, 44, 50, 17, 2], 14, 2, 64, 16, FP, 32, True, True, "nhd"),
    ([5, 2], [30, 9], 4, 4, 256, 5, BF, 256, False, True, "nhd"),
    ([5, 2], [30, 9], 4, 1, 96, 16, FP, 48, False, False, "hnd"),
    ([5, 2], [30, 9], 4, 2, 80, 16, BF, 40, False, True, "nhd"),  # half of 40 is no whole piece
    ([6], [6], 3, 3, 80, 16, BF, 80, False, True, "nhd"),
    ([4], [9], 2, 1, 33, 3, FP, 10, True, True, "nhd"),  # odd head size
    ([4], [9], 2, 1, 1, 3, FP, 0, False, True, "nhd"),
    ([8], [40], 40, 40, 64, 16, BF, 0, False, False, "nhd"),
    ([1] * 70, [i + 1 for i in range(70)], 2, 1, 64, 16, BF, 64, False, True, "nhd"),
    ([3] * 1100, [3 + i % 40 for i in range(1100)], 1, 1, 64, 16, BF, 64, False, False, "nhd"),
    ([4, 3], [9, 60], 40, 20, 128, 16, FP, 128, False, True, "hnd"),  # more head rows than a block has at once
    ([2], [7], 260, 2, 8, 16, BF, 8, True, True, "nhd"),  # more heads than the table holds
    ([5, 1], [20, 33], 3, 2, 128, 16, BF, 64, False, True, "nhd"),  # half of each head rotated
]


def tables(pr, rot, seed=1):
    g = torch.Generator().manual_seed(seed)
    n = max(pr.lens + [1])
    a = torch.rand(n, max(rot // 2, 1), generator=g) * 6.2
    w = [(1 + 0.3 * torch.randn(pr.D, generator=g)).to(pr.dtype) for _ in range(2)]
    return (torch.cat([a.cos(), a.sin()], 1) if rot else None), w


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{c[0][:3]}-{c[2]}x{c[3]}x{c[4]}-p{c[5]}-r{c[7]}{'i' if c[8] else ''}")
@pytest.mark.parametrize("in_place", [False, True])
def test_append(S, case, in_place):
    new, lens, Hq, Hkv, D, page, dtype, rot, inter, norm, layout = case
    pr = R.Problem(new, lens, Hq, Hkv, D, page, dtype, seed=D + rot, layout=layout)
    cs, (qw, kw) = tables(pr, rot)
    if not norm:
        qw = kw = None
    q, k, v = fused(pr)
    kc, vc = gpu(pr.k_cache), gpu(pr.v_cache)
    op = S.KVAppend()
    opts = dict(cos_sin=gpu(cs), interleaved=inter, q_weight=gpu(qw), k_weight=gpu(kw))
    got = op(q, k, v, kc, vc, gpu(pr.table), gpu(pr.cu), gpu(pr.kv_lens), q_out=q if in_place else None, **opts)
    torch.cuda.synchronize()
    rq, qt, rk, kt, where = R.append(pr, cs, rot, inter, qw, kw)
    assert got["status"].cpu().tolist() == [0] * pr.B
    assert ((got["q"].cpu().double() - rq).abs() <= qt).all()
    kc, vc = kc.cpu(), vc.cpu()
    want_k, want_v = pr.k_cache.double(), pr.v_cache.clone()
    tol = torch.zeros_like(want_k)
    for t, (p, s) in enumerate(where):
        want_k[p, s], tol[p, s], want_v[p, s] = rk[t], kt[t], pr.v[t]
    bits = torch.int16
    assert torch.equal(vc.contiguous().view(bits), want_v.contiguous().view(bits))
    same = torch.isnan(want_k) & torch.isnan(kc.double())
    assert (same | ((kc.double() - want_k).abs() <= tol)).all()


def test_append_bad_tokens(S):
    """Tokens without a place are not written, their q_out is zero, their sequence INVALID."""
    pr = R.Problem([4] * 6, [20, 3, 40, 30, 25, 10], 4, 2, 64, 16, BF, seed=2)
    cs, _ = tables(pr, 64)
    cs = cs[:28]  # sequences 2 and 3 run past the table of angles
    ref = R.append(pr, torch.cat([cs, torch.zeros(20, 64)]), 64)
    pr.table[4, 1] = pr.pages
    pr.kv_lens[5] = -3
    q, k, v = fused(pr)
    kc, vc = gpu(pr.k_cache), gpu(pr.v_cache)
    before = kc.clone(), vc.clone()
    got = S.KVAppend()(q, k, v, kc, vc, gpu(pr.table), gpu(pr.cu), gpu(pr.kv_lens), cos_sin=gpu(cs))
    assert got["status"].cpu().tolist() == [0, 2, 2, 2, 2, 2]
    out = got["q"].cpu().double()
    placed = [True] * 4 + [False, True, True, True] + [False] * 4 + [True, True, False, False] + [False] * 8
    for t, ok in enumerate(placed):
        if ok:
            assert ((out[t] - ref[0][t]).abs() <= ref[1][t]).all(), t
            p, s = ref[4][t]
            assert torch.equal(vc[p, s].cpu(), pr.v[t])
            before[0][p, s], before[1][p, s] = kc[p, s], vc[p, s]
        else:
            assert (out[t] == 0).all(), t
    for x, y in zip((kc, vc), before):  # nothing else was touched
        assert torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16))


@pytest.mark.parametrize("D", [128, 127])  # in 16-byte pieces, and element by element
def test_append_far_offsets(S, D):
    """Pages past 2^31 elements of a cache."""
    page, Hkv = 128, 128
    pages = (1 << 31) // (page * Hkv * D) + 4
    kc, vc = (torch.zeros(pages, page, Hkv, D, dtype=BF, device="cuda") for _ in range(2))
    pr = R.Problem([3], [130], 2, Hkv, D, page, BF, seed=3)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    assert (pages - 2) * kc.stride(0) > 1 << 31
    q, k, v = fused(pr)
    got = S.KVAppend()(q, k, v, kc, vc, table, gpu(pr.cu), gpu(pr.kv_lens))
    assert got["status"].tolist() == [0] and torch.equal(got["q"], q)
    for t, (p, slot) in enumerate([(pages - 1, 127), (pages - 2, 0), (pages - 2, 1)]):
        assert torch.equal(kc[p, slot], k[t]) and torch.equal(vc[p, slot], v[t])
        kc[p, slot] = vc[p, slot] = 0
    assert not kc.any() and not vc.any()


def test_append_statuses_without_tokens(S):
    pr = R.Problem([0, 0, 0], [5, 0, 9], 2, 1, 64, 16, BF)
    q, k, v = fused(pr)
    got = S.KVAppend()(q, k, v, gpu(pr.k_cache), gpu(pr.v_cache), gpu(pr.table), gpu(pr.cu), gpu(pr.kv_lens))
    assert got["status"].cpu().tolist() == [0, 0, 0]


# ----------------------------------------------------------------------------- verify

def softmax_rows(rng, n, V, sharp):
    z = rng.standard_normal((n, V)) * sharp
    e = np.exp(z - z.max(1, keepdims=True))
    return (e / e.sum(1, keepdims=True)).astype(np.float32)


def run_verify(S, target, draft, x, cu, u, ul, most, dtype=torch.float32, pad=0):
    def rows(a):
        if a is None:
            return None
        t = torch.zeros(a.shape[0], a.shape[1] + pad, dtype=dtype, device="cuda")
        t[:, :a.shape[1]] = torch.from_numpy(a).cuda()
        return t[:, :a.shape[1]]

    def up(a, dt):
        return torch.from_numpy(np.asarray(a, dt)).cuda()

    got = S.DraftVerifier()(rows(target), up(x, np.int32), up(cu, np.int32), up(u, np.float32), up(ul, np.float32),
                            max_draft=most, draft_probs=rows(draft))
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in got.items()}


def rounded(a, dtype):
    return a if a is None or dtype == torch.float32 else torch.from_numpy(a).to(dtype).float().numpy()


@pytest.mark.parametrize("V,dtype,has_draft,pad", [
    (1, torch.float32, True, 0), (2, torch.float32, False, 0), (37, BF, True, 0), (1000, torch.float32, True, 3),
    (1001, torch.float32, True, 0), (1003, BF, False, 0), (1003, BF, True, 2), (4096, BF, True, 0),
    (9001, torch.float32, False, 0)])
def test_verify(S, V, dtype, has_draft, pad):
    rng = np.random.default_rng(V)
    new = [0, 3, 1, 7, 0, 2, 5, 4, 4, 4]
    cu = np.concatenate([[0], np.cumsum(new)])
    N, B = int(cu[-1]), len(new)
    target = rounded(softmax_rows(rng, N + B, V, 2.0), dtype)
    draft = rounded(softmax_rows(rng, N, V, 2.0), dtype) if has_draft else None
    x = rng.integers(0, V, N)
    for b in range(B):  # likely tokens for some requests, so that runs of acceptances occur
        for i in range(new[b]):
            if b % 2:
                x[cu[b] + i] = int(target[cu[b] + b + i].argmax())
    u, ul = rng.random(N, dtype=np.float32), rng.random(B, dtype=np.float32)
    u[cu[6]:cu[7]] = 0.0
    ul[0], ul[1] = 0.0, np.float32(1) - np.float32(2.0 ** -24)
    tokens, accepted = R.verify(target, draft, x, cu, u, ul, 7)
    got = run_verify(S, target, draft, x, cu, u, ul, 7, dtype, pad)
    assert got["status"].tolist() == [0] * B
    assert np.array_equal(got["accepted"], accepted)
    assert np.array_equal(got["tokens"], tokens)


@pytest.mark.parametrize("V,B,dtype", [(151936, 3, torch.float32), (151936, 64, torch.float32), (151936, 100, BF),
                                       (50257, 200, torch.float32), (50257, 160, BF), (262144, 2, torch.float32),
                                       (262143, 160, torch.float32)])
def test_verify_full_vocabulary_split(S, V, B, dtype):
    """Thresholds that fall in every slice and warp of a large row, for every cluster size; rows
    that begin anywhere in a vector."""
    rng = np.random.default_rng(3)
    p = rounded(softmax_rows(rng, 1, V, 1.0), dtype)
    target = np.repeat(p, B, 0)
    ul = ((np.arange(B) + 0.5) / B).astype(np.float32)
    got = run_verify(S, target, None, [], [0] * (B + 1), [], ul, 0, dtype)
    w = np.floor(p[0].astype(np.float64) * 2.0 ** 40).astype(np.int64)
    c = np.cumsum(w)
    want = [int(np.searchsorted(c, int(math.floor(float(a) * 2.0 ** 31)) * int(c[-1]) >> 31, side="right")) for a in ul]
    assert got["tokens"][:, 0].tolist() == want


@pytest.mark.parametrize("V,dtype", [(151936, torch.float32), (50257, torch.float32), (50257, BF)])
def test_verify_full_vocabulary_residual(S, V, dtype):
    """The weights left above a draft's row, where the two rows are aligned differently."""
    B = 6
    rng = np.random.default_rng(4)
    target, draft = (rounded(softmax_rows(rng, n, V, 1.0), dtype) for n in (2 * B, B))
    x, u, ul = rng.integers(0, V, B), np.full(B, 0.99999, np.float32), rng.random(B, dtype=np.float32)
    u[0] = 0.0
    got = run_verify(S, target, draft, x, np.arange(B + 1), u, ul, 1, dtype)
    P, Q = (np.floor(a.astype(np.float64) * 2.0 ** 40).astype(np.int64) for a in (target, draft))
    for b in range(B):
        # both factors have 24 bits: the product is exact in 64
        ok = float(u[b]) * float(draft[b, x[b]]) < float(target[2 * b, x[b]])
        w = P[2 * b + 1] if ok else np.maximum(P[2 * b] - Q[b], 0)
        c = np.cumsum(w)
        k = int(math.floor(float(ul[b]) * 2.0 ** 31)) * int(c[-1]) >> 31
        t = int(np.searchsorted(c, k, side="right"))
        assert got["tokens"][b].tolist() == ([int(x[b]), t] if ok else [t, -1]), b


@pytest.mark.parametrize("has_draft", [False, True])
def test_verify_far_rows(S, has_draft):
    """Rows of probabilities past 2^31 elements: the last requests of a batch draw from theirs."""
    V, B = 131072, 8400
    target = torch.zeros(2 * B, V, dtype=BF, device="cuda")  # 2.2e9 elements
    x = torch.arange(B, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    rows = torch.arange(B, device="cuda")
    target[2 * rows, rows + 5] = 1.0      # never the drafted token
    target[2 * rows + 1, rows + 9] = 1.0
    last = rows >= B - 3
    target[2 * rows[last], rows[last] + 5] = 0.5  # the last three requests may keep theirs
    target[2 * rows[last], rows[last]] = 0.5
    draft = None
    if has_draft:
        draft = torch.zeros(B, V, dtype=BF, device="cuda")
        draft[rows, rows] = 1.0
    u = torch.full((B,), 0.25, device="cuda")
    got = S.DraftVerifier()(target, x, cu, u, u.clone(), max_draft=1, draft_probs=draft)
    assert not got["status"].any()
    assert torch.equal(got["accepted"], last.to(torch.int32))
    first = torch.where(last, rows, rows + 5)
    second = torch.where(last, rows + 9, -torch.ones_like(rows))
    assert torch.equal(got["tokens"].long(), torch.stack([first, second], 1))


def test_verify_edges(S):
    V = 8
    eye = np.eye(V, dtype=np.float32)
    # greedy rows: accept on the same token, else draw it; all weights above the draft zero -> p
    got = run_verify(S, eye[[3, 5, 2, 2]], eye[[3, 2]], [3, 1], [0, 1, 2], [0.9, 0.9], [0.5, 0.5], 2)
    assert got["tokens"].tolist() == [[3, 5, -1], [2, -1, -1]] and got["accepted"].tolist() == [1, 0]
    # a refused token (u q = p, not below) whose row equals the draft's: drawn from p
    half = np.full((1, V), 0.125, np.float32)
    got = run_verify(S, np.repeat(half * 0.5, 2, 0), half, [4], [0, 1], [0.5], [0.0], 1)
    assert got["tokens"].tolist() == [[0, -1]] and got["status"].tolist() == [0]
    # zero probability is refused with any number, also 0
    got = run_verify(S, eye[[3, 3]], None, [1], [0, 1], [0.0], [0.99], 1)
    assert got["tokens"].tolist() == [[3, -1]]


def test_verify_bad_requests(S):
    V, B = 50, 12
    rng = np.random.default_rng(9)

    def make():
        return (softmax_rows(rng, 2 * B + B, V, 1.0), softmax_rows(rng, 2 * B, V, 1.0), rng.integers(0, V, 2 * B),
                np.arange(0, 2 * B + 1, 2), np.full(2 * B, 0.999, np.float32), rng.random(B, dtype=np.float32))

    target, draft, x, cu, u, ul = make()
    good = run_verify(S, target, draft, x, cu, u, ul, 2)
    assert good["status"].tolist() == [0] * B
    t2, x2, u2, ul2 = target.copy(), x.copy(), u.copy(), ul.copy()
    x2[0] = V
    x2[2 * 1 + 1] = -1
    u2[2 * 2] = 1.0
    u2[2 * 3] = np.nan
    ul2[4] = -0.1
    ul2[5] = np.inf
    a6 = good["accepted"][6]
    t2[3 * 6 + a6, 7] = np.nan
    a7 = good["accepted"][7]
    t2[3 * 7 + a7, 49] = -0.25
    t2[3 * 8:3 * 9] = 0.0  # no mass
    a9 = good["accepted"][9]
    t2[3 * 9 + a9, 0] = 1.5
    got = run_verify(S, t2, draft, x2, cu, u2, ul2, 2)
    assert got["status"].tolist() == [2] * 10 + [0, 0]
    assert (got["tokens"][:10] == -1).all() and (got["accepted"][:10] == 0).all()
    assert np.array_equal(got["tokens"][10:], good["tokens"][10:])
    # offsets out of order, past the end, more drafted than allowed
    cu2 = cu.copy()
    cu2[3] = 3
    cu2[-1] = 2 * B + 5
    got = run_verify(S, target, draft, x, cu2, u, ul, 2)
    assert got["status"][2] == 2 and got["status"][3] == 2 and got["status"][-1] == 2
    assert got["status"][:2].tolist() == [0, 0]
    assert run_verify(S, target, draft, x, cu, u, ul, 1)["status"].tolist() == [2] * B


@pytest.mark.parametrize("B", [3, 100, 300])  # every cluster size
def test_verify_bad_first_and_last_probabilities(S, B):
    """A probability out of range that a warp meets first of all, or last: the request is INVALID
    as a whole and its neighbours are what they were, call after call."""
    V = 5000
    rng = np.random.default_rng(B)
    target = softmax_rows(rng, B, V, 1.0)
    ul = rng.random(B, dtype=np.float32)
    good = run_verify(S, target, None, [], [0] * (B + 1), [], ul, 0)
    assert good["status"].tolist() == [0] * B
    broken = target.copy()
    broken[0::3, 0] = 1.5
    broken[1::3, V - 1] = np.nan
    for _ in range(20):
        got = run_verify(S, broken, None, [], [0] * (B + 1), [], ul, 0)
        want = np.where(np.arange(B) % 3 == 2, good["tokens"][:, 0], -1)
        assert got["status"].tolist() == [0 if b % 3 == 2 else 2 for b in range(B)]
        assert np.array_equal(got["tokens"][:, 0], want)


def test_verify_keeps_the_target_distribution(S):
    """First token of a verification, over many requests with one drafted token each drawn
    from q, is distributed as p: chi-square with 7 degrees of freedom below its 1e-6 point."""
    V, B = 8, 40000
    rng = np.random.default_rng(21)
    p, q = softmax_rows(rng, 1, V, 1.0), softmax_rows(rng, 1, V, 1.0)
    x = rng.choice(V, size=B, p=(q[0].astype(np.float64) / q[0].astype(np.float64).sum()))
    got = run_verify(S, np.repeat(p, 2 * B, 0), np.repeat(q, B, 0), x, np.arange(B + 1),
                     rng.random(B, dtype=np.float32), rng.random(B, dtype=np.float32), 1)
    seen = np.bincount(got["tokens"][:, 0], minlength=V)
    want = p[0].astype(np.float64) / p[0].astype(np.float64).sum() * B
    assert ((seen - want) ** 2 / want).sum() < 43.0


def test_verify_refusals(S):
    V = 10
    t = torch.full((3, V), 0.1, device="cuda")
    x = torch.zeros(2, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    u, ul = torch.zeros(2, device="cuda"), torch.zeros(1, device="cuda")
    op = S.DraftVerifier()
    op(t, x, cu, u, ul, max_draft=2)
    for bad in ((t.double(), x, cu, u, ul), (t[:2], x, cu, u, ul), (t, x.long(), cu, u, ul), (t, x, cu[:1], u, ul),
                (t, x, cu, u[:1], ul), (t.cpu(), x, cu, u, ul)):
        with pytest.raises(ValueError):
            op(*bad, max_draft=2)
    with pytest.raises(ValueError):
        op(t, x, cu, u, ul, max_draft=2, draft_probs=t)
    with pytest.raises(Exception) as e:
        op(t, x, cu, u, ul, max_draft=-1)
    assert isinstance(e.value, (ValueError, RuntimeError))


# ----------------------------------------------------------------------------- together

def test_example_step(S):
    """The example's loop: verified tokens are those of the rule on the probabilities that the
    step used, and logits of a chunk equal those of its tokens one by one on a second cache
    within the rounding of the chunk's bf16 activations."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_step.py")
    spec = importlib.util.spec_from_file_location("speculative_step", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    B, V, k = 3, 500, 3
    shape = dict(vocab=V, Hq=4, Hkv=2, D=64, batch=B, max_len=128)
    target, draft = ex.Decoder(layers=2, seed=0, **shape), ex.Decoder(layers=1, seed=0, **shape)
    loop = ex.SpeculativeLoop(target, draft, V, B, k)
    loop.prefill([[1, 2, 3, 4], [5] * 20, list(range(40, 97))])
    for _ in range(5):
        before = loop.lens.clone()
        out = loop.step()
        torch.cuda.synchronize()
        used = {n: t.cpu().numpy() if torch.is_tensor(t) else t for n, t in loop.used.items()}
        tokens, accepted = R.verify(used["target_probs"], used["draft_probs"], used["draft_tokens"], used["cu_draft"],
                                    used["u_accept"], used["u_sample"], k)
        assert np.array_equal(out["tokens"].cpu().numpy(), tokens)
        assert np.array_equal(out["accepted"].cpu().numpy(), accepted)
        assert torch.equal(loop.lens.cpu(), before.cpu() + 1 + torch.from_numpy(accepted))
    # the same weights, one token at a time
    chunk, single = ex.Decoder(layers=2, seed=3, **shape), ex.Decoder(layers=2, seed=3, **shape)
    n = 40
    ids = torch.randint(0, V, (B, n), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    got = chunk(ids.reshape(-1).contiguous(), one * n, torch.full((B,), n, dtype=torch.int32, device="cuda"), n)
    got = got.view(B, n, V)
    for i in range(n):
        want = single(ids[:, i].contiguous(), one, torch.full((B,), i + 1, dtype=torch.int32, device="cuda"), 1)
        # both round their activations to bf16 (2^-8) some twenty times along the two layers;
        # such errors add up like their square root, and a logit is a sum over the row
        size = want.norm(dim=1, keepdim=True) / V ** 0.5
        assert ((got[:, i] - want).abs() <= 8 * 2.0 ** -8 * 20 ** 0.5 * size).all(), i


def test_example_prompts_of_one_token(S):
    """Prompts whose only token is left for the first step: nothing is prefilled."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_step.py")
    spec = importlib.util.spec_from_file_location("speculative_step", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    B, V = 2, 300
    shape = dict(vocab=V, Hq=4, Hkv=2, D=64, batch=B, max_len=64)
    loop = ex.SpeculativeLoop(ex.Decoder(layers=2, **shape), ex.Decoder(layers=1, **shape), V, B, 2)
    loop.prefill([[7], [11]])
    for _ in range(3):
        out = loop.step()
        assert not out["status"].any()
        assert ((out["tokens"] >= 0).sum(1) == out["accepted"] + 1).all()
    assert (loop.lens >= 3).all()
