"""Layout and host-side refusals of the tree-step and page entry points.  No GPU needed."""
import ctypes
import os
import random
import subprocess
import tempfile
import types

import numpy as np
import pytest

import tree_reference as TR

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from constrained_logits_sampling_gb300 import build, sampler
    build.build()
    return sampler.load_library()


def structs():
    from constrained_logits_sampling_gb300 import pages as G, tree as S
    return [("clsample_tree_plan_args_t", S.TreePlanArgs), ("clsample_tree_mask_t", S.TreeMask),
            ("clsample_verify_tree_args_t", S.VerifyTreeArgs), ("clsample_keep_path_args_t", G.KeepPathArgs),
            ("clsample_copy_pages_args_t", G.CopyPagesArgs), ("clsample_page_pool_t", G.PoolArgs),
            ("clsample_page_batch_t", G.BatchArgs)]


def test_args_layouts_match_header(lib):
    body = ""
    for name, cls in structs():
        body += f'  printf("{name} %zu\\n", sizeof({name}));\n'
        for f, _ in cls._fields_:
            body += f'  printf("{name}.{f} %zu\\n", offsetof({name}, {f}));\n'
    src = ('#include <stdio.h>\n#include <stddef.h>\n#include "clsample.h"\nint main(void){\n' + body + "  return 0;\n}\n")
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "probe.c"), os.path.join(d, "probe")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", exe, c], check=True)
        got = dict(line.split() for line in subprocess.run([exe], capture_output=True, text=True,
                                                           check=True).stdout.splitlines())
    for name, cls in structs():
        assert int(got[name]) == ctypes.sizeof(cls), name
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)


def filled(cls, pointers, **kw):
    a = cls(**kw)
    for n in pointers:
        setattr(a, n, 16 * (1 + pointers.index(n)))
    return a


def changed(a, change):
    for k, v in change.items():
        setattr(a, k, v)
    return a


def plan(**change):
    from constrained_logits_sampling_gb300.tree import TreePlanArgs
    return changed(filled(TreePlanArgs, ["parents", "cu_draft", "kv_lens", "mask"], B=1, N=3, max_draft=40, mask_stride=2),
                   change)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), -2), (dict(N=-1), -2), (dict(max_draft=-1), -9), (dict(max_draft=1024), -9), (dict(window=-1), -9),
    (dict(mask_stride=1), -4), (dict(parents=None), -1), (dict(cu_draft=None), -1), (dict(kv_lens=None), -1),
    (dict(mask=None), -1)])
def test_plan_refusals(lib, change, code):
    assert lib.clsample_tree_plan(ctypes.byref(plan(**change)), None) == code


def verify(**change):
    from constrained_logits_sampling_gb300.tree import VerifyTreeArgs
    return changed(filled(VerifyTreeArgs, ["target", "draft", "draft_rows", "draft_tokens", "parents", "cu_draft", "u_accept",
                                           "u_sample", "tokens", "path"], B=1, N=3, V=100, dtype=0, max_draft=3, max_path=2,
                          draft_rows_count=3, target_stride=100, draft_stride=100, token_stride=3, path_stride=2), change)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), -2), (dict(N=-1), -2), (dict(V=0), -3), (dict(V=262145), -3), (dict(dtype=5), -5), (dict(max_draft=-1), -9),
    (dict(max_draft=1024), -9), (dict(max_path=4), -9), (dict(max_path=-1), -9), (dict(draft_rows_count=-1), -9),
    (dict(target_stride=99), -4), (dict(draft_stride=99), -4), (dict(token_stride=2), -4), (dict(path_stride=1), -4),
    (dict(target=None), -1), (dict(draft_tokens=None), -1), (dict(parents=None), -1), (dict(cu_draft=None), -1),
    (dict(u_accept=None), -1), (dict(u_sample=None), -1), (dict(tokens=None), -1)])
def test_verify_refusals(lib, change, code):
    assert lib.clsample_verify_tree(ctypes.byref(verify(**change)), None) == code


def keep(**change):
    from constrained_logits_sampling_gb300.pages import KeepPathArgs
    return changed(filled(KeepPathArgs, ["k_cache", "v_cache", "page_table", "cu_draft", "kv_lens", "path", "accepted",
                                         "new_lens"], B=1, N=3, layers=1, Hkv=2, D=64, dtype=0, num_pages=4, page_size=16,
                          max_pages=2, max_path=3, table_stride=2, path_stride=3), change)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), -2), (dict(N=-1), -2), (dict(dtype=2), -5), (dict(layers=0), -9), (dict(Hkv=0), -9), (dict(D=0), -9),
    (dict(D=257), -9), (dict(num_pages=-1), -9), (dict(page_size=0), -9), (dict(max_pages=-1), -9), (dict(max_path=1024), -9),
    (dict(max_path=-1), -9), (dict(layers=1 << 20, Hkv=16), -9), (dict(table_stride=1), -4), (dict(path_stride=2), -4),
    (dict(k_cache=None), -1), (dict(v_cache=None), -1), (dict(page_table=None), -1), (dict(cu_draft=None), -1),
    (dict(kv_lens=None), -1), (dict(path=None), -1), (dict(accepted=None), -1), (dict(new_lens=None), -1),
    (dict(new_lens=80), -9)])  # kv_lens itself
def test_keep_refusals(lib, change, code):
    assert lib.clsample_keep_path(ctypes.byref(keep(**change)), None) == code


def copy(**change):
    from constrained_logits_sampling_gb300.pages import CopyPagesArgs
    return changed(filled(CopyPagesArgs, ["k_cache", "v_cache", "copies"], n=1, layers=1, Hkv=2, D=64, dtype=0, num_pages=4,
                          page_size=16), change)


@pytest.mark.parametrize("change,code", [
    (dict(n=-1), -2), (dict(dtype=2), -5), (dict(layers=0), -9), (dict(Hkv=0), -9), (dict(D=257), -9), (dict(num_pages=-1), -9),
    (dict(page_size=0), -9), (dict(copies=None), -1), (dict(k_cache=None), -1), (dict(v_cache=None), -1)])
def test_copy_refusals(lib, change, code):
    assert lib.clsample_copy_pages(ctypes.byref(copy(**change)), None) == code


def pool(pool_change=(), batch_change=()):
    from constrained_logits_sampling_gb300.pages import BatchArgs, PoolArgs
    p = filled(PoolArgs, ["refs", "free_bits", "stamps", "epoch", "list"], num_pages=8, page_size=4)
    b = filled(BatchArgs, ["page_table", "held", "kv_lens"], B=2, max_pages=3, table_stride=3)
    return changed(p, dict(pool_change)), changed(b, dict(batch_change))


POOL = [(dict(num_pages=-1), {}, -9), (dict(num_pages=(1 << 30) + 1), {}, -9), (dict(page_size=0), {}, -9),
        (dict(refs=None), {}, -1), (dict(free_bits=None), {}, -1), (dict(stamps=None), {}, -1), (dict(epoch=None), {}, -1),
        (dict(list=None), {}, -1), ({}, dict(B=-1), -2), ({}, dict(max_pages=-1), -9), ({}, dict(table_stride=2), -4),
        ({}, dict(held=None), -1), ({}, dict(kv_lens=None), -1), ({}, dict(page_table=None), -1)]


@pytest.mark.parametrize("pc,bc,code", POOL)
def test_pool_refusals(lib, pc, bc, code):
    p, b = (ctypes.byref(x) for x in pool(pc, bc))
    assert lib.clsample_pages_fork(p, b, 16, 32, 1, None, None) == code
    assert lib.clsample_pages_reserve(p, b, 16, 32, None, None, None) == code
    assert lib.clsample_pages_trim(p, b, None, None) == code


def test_pool_call_refusals(lib):
    p, b = (ctypes.byref(x) for x in pool())
    for null in ((None, b), (p, None)):
        assert lib.clsample_pages_trim(*null, None, None) == -1
    assert lib.clsample_pages_fork(p, b, 16, 32, -1, None, None) == -2
    assert lib.clsample_pages_fork(p, b, None, 32, 1, None, None) == -1
    assert lib.clsample_pages_fork(p, b, 16, None, 1, None, None) == -1
    assert lib.clsample_pages_reserve(p, b, None, 32, None, None, None) == -1
    assert lib.clsample_pages_reserve(p, b, 16, None, None, None, None) == -1


def test_nothing_to_do(lib):
    for name in ("clsample_tree_plan", "clsample_verify_tree", "clsample_keep_path", "clsample_copy_pages"):
        assert getattr(lib, name)(None, None) == -1
    assert lib.clsample_tree_plan(ctypes.byref(plan(B=0)), None) == 0
    assert lib.clsample_verify_tree(ctypes.byref(verify(B=0)), None) == 0
    assert lib.clsample_keep_path(ctypes.byref(keep(B=0)), None) == 0
    assert lib.clsample_copy_pages(ctypes.byref(copy(n=0)), None) == 0
    p, b = (ctypes.byref(x) for x in pool())
    assert lib.clsample_pages_fork(p, b, 16, 32, 0, None, None) == 0
    p, b = (ctypes.byref(x) for x in pool({}, dict(B=0)))
    assert lib.clsample_pages_trim(p, b, None, None) == 0
    assert lib.clsample_pages_reserve(p, b, None, None, None, None, None) == 0


def test_tree_attention_null(lib):
    from constrained_logits_sampling_gb300.speculative import AttentionArgs
    from constrained_logits_sampling_gb300.tree import TreeMask
    a, m = AttentionArgs(), TreeMask()
    assert lib.clsample_tree_attention(None, ctypes.byref(a), ctypes.byref(m), None) == -1
    assert lib.clsample_tree_attention(16, ctypes.byref(a), None, None) == -1
    assert lib.clsample_tree_attention(16, None, ctypes.byref(m), None) == -1
    assert lib.clsample_kv_append_at(None, None, None) == -1


@pytest.mark.parametrize("where,name,function", [
    ("tree", "TreePlan", "clsample_tree_plan"), ("tree", "TreeVerifier", "clsample_verify_tree"),
    ("pages", "KeepPath", "clsample_keep_path"), ("pages", "CopyPages", "clsample_copy_pages"),
    ("pages", "PagePool", "clsample_pages_trim")])
def test_calls_while_another_device_is_current(lib, monkeypatch, where, name, function):
    """An object's tensors are its own device's: with another device current nothing is launched."""
    import importlib

    import torch
    M = importlib.import_module(f"constrained_logits_sampling_gb300.{where}")
    calls = []
    op = getattr(M, name).__new__(getattr(M, name))
    op._L = types.SimpleNamespace(**{function: lambda *a: calls.append(a) or 0})
    op.device = torch.device("cuda", 0)
    monkeypatch.setattr(M, "_stream_ptr", lambda stream: 0)
    if name == "PagePool":
        op._args = M.PoolArgs()
        args = M._PoolCall(function, op._args, M.BatchArgs(), (None,), ())
    else:
        args = {"TreePlan": plan, "TreeVerifier": verify, "KeepPath": keep, "CopyPages": copy}[name]()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(RuntimeError) as e:
        op.apply(args)
    assert e.value.code == -7 and not calls
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    op.apply(args)
    assert len(calls) == 1


@pytest.mark.parametrize("index", range(7))
def test_numbers_past_32_bits_are_refused(lib, index):
    from constrained_logits_sampling_gb300.speculative import _I32
    _, cls = structs()[index]
    a = cls()
    for field in (n for n, t in cls._fields_ if t is _I32):
        for value in ((1 << 32) + 5, 1 << 31, -(1 << 31) - 1):
            with pytest.raises(ValueError):
                setattr(a, field, value)
        setattr(a, field, (1 << 31) - 1)


def test_reference_pool_keeps_its_books():
    """The plain pool that the device's is held to: what its tables name is what it counts."""
    r = random.Random(4)
    p = TR.Pool(30, 4, 6, 10)
    for _ in range(300):
        kind = r.randrange(3)
        if kind == 0:
            new = [r.choice([0, 1, 5]) for _ in range(6)]
            if not any(p.reserve(new)[1]):
                p.lens = [m + n for m, n in zip(p.lens, new)]
        elif kind == 1:
            p.fork([r.randrange(6)], [r.randrange(6)])
        else:
            p.lens = [m if r.random() < 0.7 else r.randint(0, m) for m in p.lens]
            p.trim()
        count = [0] * 30
        for b in range(6):
            for k in range(p.held[b]):
                count[p.table[b][k]] += 1
        assert count == p.refs


def test_reference_walk_of_a_chain_is_the_chains():
    import spec_reference as R
    rng = np.random.default_rng(1)
    for draft in (True, False):
        target = rng.dirichlet(np.ones(9), 12).astype(np.float32)
        q = rng.dirichlet(np.ones(9), 9).astype(np.float32) if draft else None
        x, cu = rng.integers(0, 9, 9), np.array([0, 4, 4, 9])
        u, ul = rng.random(9, np.float32), rng.random(3, np.float32)
        parents = TR.chain(4) + TR.chain(5)
        tokens, path, accepted = TR.verify_tree(target, q, np.arange(9), x, parents, cu, u, ul, 5)
        want, count = R.verify(target, q, x, cu, u, ul, 5)
        assert np.array_equal(tokens, want) and np.array_equal(accepted, count)
        assert all(list(path[b, :accepted[b]]) == list(range(accepted[b])) for b in range(3))
