"""The 4-bit cache's entry points and the head norms refuse what they cannot do before anything is launched (CPU: no
device is touched)."""
import math

import pytest
import torch

import chunked_prefill_paged_slot_gb300 as cpsa
from test_rope_append_refusals import BAD

OK, NULL, SHAPE, ALIGN, UNSUP, NODEV = 0, -1, -2, -3, -4, -7
A = 0x10000          # an aligned address that is never read
APPENDS = {"cpp_rope_kv_cache_write_q4": (4, False), "cpp_norm_rope_kv_cache_write": (16, True),
           "cpp_norm_rope_kv_cache_write_q8": (8, True), "cpp_norm_rope_kv_cache_write_q4": (4, True)}


def append(name, **over):
    bits, norm = APPENDS[name]
    a = dict(q=A, k=A, v=A, qs=4 * 64, ks=2 * 64, vs=2 * 64)
    if norm:
        a.update(qw=A, kw=A, eps=1e-6)
    a.update(pos=A, cs=A, top=100, rot=64, inter=0, slots=A, T=3, Hq=4, Hkv=2, d=64, P=16, pages=8, out=A + 4096, kc=A, vc=A)
    if bits < 16:
        a.update(ksc=A, vsc=A)
    a.update(err=A, stream=None)
    assert set(over) <= set(a), over
    a.update(over)
    return getattr(cpsa.load(), name)(*a.values())


@pytest.mark.parametrize("name", APPENDS)
@pytest.mark.parametrize("over,status", BAD, ids=lambda x: str(x))
def test_appends_refuse(name, over, status):
    assert append(name, **over) == status


@pytest.mark.parametrize("name", [n for n, (_, norm) in APPENDS.items() if norm])
@pytest.mark.parametrize("over,status", [
    (dict(eps=0.0), SHAPE), (dict(eps=-1e-6), SHAPE), (dict(eps=math.nan), SHAPE), (dict(eps=math.inf), SHAPE),
    (dict(qw=None), NULL), (dict(kw=None), NULL), (dict(qw=A + 4), ALIGN), (dict(kw=A + 8), ALIGN)], ids=str)
def test_norms_refuse(name, over, status):
    assert append(name, **over) == status


@pytest.mark.parametrize("name", [n for n, (bits, _) in APPENDS.items() if bits == 4])
@pytest.mark.parametrize("over,status", [(dict(P=4), UNSUP), (dict(P=512), UNSUP), (dict(ksc=None), NULL),
                                         (dict(vsc=None), NULL), (dict(ksc=A + 8), ALIGN), (dict(vsc=A + 4), ALIGN)], ids=str)
def test_4_bit_caches_refuse(name, over, status):
    assert append(name, **over) == status


@pytest.mark.parametrize("name", APPENDS)
def test_empty_calls_and_optional_arguments(name):
    assert append(name, T=0, q=None, k=None, v=None, slots=None, out=None, kc=None, vc=None) == OK
    if not torch.cuda.is_available():      # every check passed: the next thing is the device
        assert append(name) == NODEV
        assert append(name, rot=0, pos=None, cs=None) == NODEV
        more = dict(qw=None) if APPENDS[name][1] else {}
        assert append(name, Hq=0, q=None, out=None, qs=0, **more) == NODEV
        assert append(name, q=A, out=A) == NODEV


def read(**over):
    a = dict(kc=A, vc=A, ks=A, vs=A, slots=A, T=3, Hkv=2, d=64, P=16, pages=8, k=A, v=A, err=A, stream=None)
    assert set(over) <= set(a), over
    a.update(over)
    return cpsa.load().cpp_kv_cache_read_q4(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(Hkv=0), SHAPE), (dict(Hkv=1 << 16), SHAPE), (dict(pages=-1), SHAPE),
    (dict(pages=1 << 61), SHAPE), (dict(d=96), UNSUP), (dict(P=4), UNSUP), (dict(P=24), UNSUP), (dict(P=512), UNSUP),
    (dict(kc=None), NULL), (dict(vc=None), NULL), (dict(ks=None), NULL), (dict(vs=None), NULL), (dict(slots=None), NULL),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(err=None), NULL), (dict(kc=A + 8), ALIGN), (dict(vc=A + 4), ALIGN),
    (dict(ks=A + 8), ALIGN), (dict(vs=A + 1), ALIGN), (dict(k=A + 8), ALIGN), (dict(v=A + 2), ALIGN)], ids=str)
def test_read_refuses(over, status):
    assert read(**over) == status


def test_empty_read():
    assert read(T=0, kc=None, slots=None, k=None, v=None) == OK
    if not torch.cuda.is_available():
        assert read() == NODEV


def test_bindings_refuse_host_tensors_and_wrong_shapes():
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    held = [torch.zeros(4, 2, 16, n, dtype=torch.uint8) for n in (32, 32, 4, 4)]
    wide = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    w, err = torch.ones(64), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(cpsa.CpsaError, match="CUDA tensor"):
        cpsa.cpp_rope_kv_cache_write_q4(None, x, x, None, None, slots, *held, None, err)
    with pytest.raises(cpsa.CpsaError, match="inconsistent shapes"):      # a cache of 64 bytes a row holds 128 columns
        cpsa.cpp_rope_kv_cache_write_q4(None, x, x, None, None, slots, wide, wide, *held[2:], None, err)
    with pytest.raises(cpsa.CpsaError, match="inconsistent shapes"):
        cpsa.cpp_norm_rope_kv_cache_write(None, x, x[:2], None, w, None, None, slots, wide, wide, None, err)
    with pytest.raises(cpsa.CpsaError, match="CUDA tensor"):
        cpsa.cpp_kv_cache_read_q4(*held, slots, x, x, err)


def attn(**over):
    a = dict(q=A, kc=A, vc=A, ks=A, vs=A, ql=A, sl=A, bt=A, B=2, T=5, M=4, Hq=4, Hkv=2, d=64, P=16, pages=8, scale=0.0,
             splits=8, out=A, ws=A, wsb=1 << 30, err=A, stream=None)
    assert set(over) <= set(a), over
    a.update(over)
    return cpsa.load().cpp_chunked_prefill_attn_q4(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(ks=None), NULL), (dict(vs=None), NULL), (dict(q=None), NULL), (dict(kc=None), NULL), (dict(vc=None), NULL),
    (dict(ql=None), NULL), (dict(sl=None), NULL), (dict(bt=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL),
    (dict(err=None), NULL), (dict(B=-1), SHAPE), (dict(T=-1), SHAPE), (dict(B=0), SHAPE), (dict(M=-1), SHAPE),
    (dict(pages=-1), SHAPE), (dict(pages=1 << 40), SHAPE), (dict(splits=0), SHAPE), (dict(splits=33), SHAPE),
    (dict(q=A + 8), ALIGN), (dict(kc=A + 8), ALIGN), (dict(vc=A + 8), ALIGN), (dict(ks=A + 8), ALIGN), (dict(vs=A + 4), ALIGN),
    (dict(out=A + 2), ALIGN), (dict(ws=A + 4), ALIGN), (dict(d=96), UNSUP), (dict(P=4), UNSUP), (dict(P=24), UNSUP),
    (dict(P=512), UNSUP), (dict(Hq=5), UNSUP), (dict(Hq=34), UNSUP), (dict(wsb=100), -5)], ids=str)
def test_attention_refuses(over, status):
    assert attn(**over) == status


def test_empty_attention():
    assert attn(T=0, B=0, q=None, ks=None, vs=None) == OK
    if not torch.cuda.is_available():
        assert attn() == NODEV


def test_attention_binding_refuses_wrong_types():
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    c, sc = torch.zeros(2, 2, 16, 32, dtype=torch.uint8), torch.zeros(2, 2, 16, 4, dtype=torch.uint8)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(cpsa.CpsaError, match="k_cache must be"):
        cpsa.cpp_chunked_prefill_attn_q4(q, c, c, sc, sc, i, i, i.view(1, 1), q, c.view(-1), i)
