"""Layout and host-side refusals of the speculative-step entry points.  No GPU needed."""
import ctypes
import os
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from constrained_logits_sampling_gb300 import build, sampler
    build.build()
    return sampler.load_library()


def test_args_layouts_match_header(lib):
    from constrained_logits_sampling_gb300 import speculative as S
    pairs = [("clsample_kv_append_args_t", S.KVAppendArgs), ("clsample_attention_args_t", S.AttentionArgs),
             ("clsample_verify_args_t", S.VerifyArgs)]
    body = ""
    for name, cls in pairs:
        body += f'  printf("{name} %zu\\n", sizeof({name}));\n'
        for f, _ in cls._fields_:
            body += f'  printf("{name}.{f} %zu\\n", offsetof({name}, {f}));\n'
    src = ('#include <stdio.h>\n#include <stddef.h>\n#include "clsample.h"\nint main(void){\n' + body +
           "  return 0;\n}\n")
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "probe.c"), os.path.join(d, "probe")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", exe, c], check=True)
        got = dict(line.split() for line in subprocess.run([exe], capture_output=True, text=True,
                                                           check=True).stdout.splitlines())
    for name, cls in pairs:
        assert int(got[name]) == ctypes.sizeof(cls), name
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)


def test_new_codes_have_texts(lib):
    for code in (-9, -10):
        assert lib.clsample_strerror(code) != b"unknown error"


def _append(**kw):
    from constrained_logits_sampling_gb300.speculative import KVAppendArgs
    a = KVAppendArgs(B=1, T=1, Hq=2, Hkv=1, D=64, dtype=0, num_pages=1, page_size=16, max_pages=1, rot_dim=64,
                     max_pos=16, eps=1e-6, table_stride=1, cs_stride=64)
    for n in ("q", "k", "v", "q_out", "k_cache", "v_cache", "page_table", "cu_new", "kv_lens", "cos_sin"):
        setattr(a, n, 16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), -2), (dict(T=-1), -2), (dict(dtype=2), -5), (dict(D=0), -9), (dict(D=257), -9), (dict(Hkv=0), -9),
    (dict(page_size=0), -9), (dict(rot_dim=63), -9), (dict(rot_dim=66), -9), (dict(eps=float("nan")), -9),
    (dict(eps=-1.0), -9), (dict(table_stride=0), -4), (dict(cs_stride=63), -4), (dict(q=None), -1),
    (dict(k=None), -1), (dict(v_cache=None), -1), (dict(q_out=None), -1), (dict(cos_sin=None), -1),
    (dict(cu_new=None), -1), (dict(kv_lens=None), -1), (dict(page_table=None), -1)])
def test_append_refusals(lib, change, code):
    assert lib.clsample_kv_append(ctypes.byref(_append(**change)), None) == code


def test_append_nothing_to_do(lib):
    assert lib.clsample_kv_append(None, None) == -1
    assert lib.clsample_kv_append(ctypes.byref(_append(B=0)), None) == 0
    assert lib.clsample_kv_append(ctypes.byref(_append(T=0)), None) == 0


def test_attention_handle_refusals(lib):
    from constrained_logits_sampling_gb300.speculative import AttentionArgs
    assert lib.clsample_attention_create(None) == -1
    assert lib.clsample_chunk_attention(None, ctypes.byref(AttentionArgs()), None) == -1
    lib.clsample_attention_destroy(None)


def _verify(**kw):
    from constrained_logits_sampling_gb300.speculative import VerifyArgs
    a = VerifyArgs(B=1, N=2, V=100, dtype=0, max_draft=2, target_stride=100, draft_stride=100, token_stride=3)
    for n in ("target", "draft", "draft_tokens", "cu_draft", "u_accept", "u_sample", "tokens"):
        setattr(a, n, 16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), -2), (dict(N=-1), -2), (dict(V=0), -3), (dict(V=262145), -3), (dict(dtype=7), -5),
    (dict(max_draft=-1), -9), (dict(target_stride=99), -4), (dict(draft_stride=99), -4), (dict(token_stride=2), -4),
    (dict(target=None), -1), (dict(draft_tokens=None), -1), (dict(u_accept=None), -1), (dict(u_sample=None), -1),
    (dict(tokens=None), -1), (dict(cu_draft=None), -1)])
def test_verify_refusals(lib, change, code):
    assert lib.clsample_verify(ctypes.byref(_verify(**change)), None) == code


def test_verify_nothing_to_do(lib):
    assert lib.clsample_verify(None, None) == -1
    assert lib.clsample_verify(ctypes.byref(_verify(B=0)), None) == 0


@pytest.mark.parametrize("name,function", [("KVAppend", "clsample_kv_append"), ("DraftVerifier", "clsample_verify")])
def test_calls_while_another_device_is_current(lib, monkeypatch, name, function):
    """An object's tensors are its own device's: with another device current nothing is launched."""
    import types

    import torch
    from constrained_logits_sampling_gb300 import speculative as S
    calls = []
    op = getattr(S, name).__new__(getattr(S, name))
    op._L = types.SimpleNamespace(**{function: lambda *a: calls.append(a) or 0})
    op.device = torch.device("cuda", 0)
    monkeypatch.setattr(S, "_stream_ptr", lambda stream: 0)
    args = (S.KVAppendArgs if name == "KVAppend" else S.VerifyArgs)()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(RuntimeError) as e:
        op.apply(args)
    assert e.value.code == -7 and not calls
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    op.apply(args)
    assert len(calls) == 1


@pytest.mark.parametrize("cls,field", [("AttentionArgs", "window"), ("AttentionArgs", "max_new"), ("AttentionArgs", "T"),
                                       ("KVAppendArgs", "rot_dim"), ("KVAppendArgs", "T"), ("VerifyArgs", "max_draft"),
                                       ("VerifyArgs", "N")])
def test_numbers_past_32_bits_are_refused(lib, cls, field):
    """A window of 2^32 + 5 is not one of 5."""
    from constrained_logits_sampling_gb300 import speculative as S
    a = getattr(S, cls)()
    for value in ((1 << 32) + 5, 1 << 31, -(1 << 31) - 1, 1 << 70):
        with pytest.raises(ValueError):
            setattr(a, field, value)
        assert getattr(a, field) == 0
    for value in ((1 << 31) - 1, -(1 << 31), 7):
        setattr(a, field, value)
        assert getattr(a, field) == value
    a.page_stride = a.target_stride = 1 << 40  # 64-bit fields, or none of the structure's
    assert getattr(a, "page_stride") == 1 << 40
