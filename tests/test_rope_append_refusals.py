"""The rotary appends refuse what they cannot do before anything is launched (CPU: no device is touched)."""
import pytest
import torch

import chunked_prefill_paged_slot_gb300 as cpsa

OK, NULL, SHAPE, ALIGN, UNSUP, NODEV = 0, -1, -2, -3, -4, -7
A = 0x10000          # an aligned address that is never read


def call(q8, **over):
    a = dict(q=A, k=A, v=A, qs=4 * 64, ks=2 * 64, vs=2 * 64, pos=A, cs=A, top=100, rot=64, inter=0, slots=A, T=3, Hq=4,
             Hkv=2, d=64, P=16, pages=8, out=A + 4096, kc=A, vc=A)
    if q8:
        a.update(ksc=A, vsc=A)
    a.update(err=A, stream=None)
    assert set(over) <= set(a), over
    a.update(over)
    fn = cpsa.load().cpp_rope_kv_cache_write_q8 if q8 else cpsa.load().cpp_rope_kv_cache_write
    return fn(*a.values())


BAD = [
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(Hkv=0), SHAPE), (dict(Hq=-1), SHAPE), (dict(pages=-1), SHAPE),
    (dict(pages=1 << 61), SHAPE), (dict(top=-1), SHAPE), (dict(rot=-16), SHAPE),
    (dict(qs=4 * 64 - 8), SHAPE), (dict(ks=64), SHAPE), (dict(vs=0), SHAPE), (dict(ks=-128), SHAPE),
    (dict(qs=1 << 40), SHAPE), (dict(q=A, out=A, qs=512), SHAPE),
    (dict(d=96), UNSUP), (dict(d=256), UNSUP), (dict(rot=80), UNSUP), (dict(rot=8), UNSUP), (dict(rot=24), UNSUP),
    (dict(P=24), UNSUP), (dict(P=0), UNSUP), (dict(P=1 << 21), UNSUP),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(q=None), NULL), (dict(out=None), NULL), (dict(slots=None), NULL),
    (dict(pos=None), NULL), (dict(cs=None), NULL), (dict(kc=None), NULL), (dict(vc=None), NULL), (dict(err=None), NULL),
    (dict(k=A + 8), ALIGN), (dict(v=A + 2), ALIGN), (dict(q=A + 8), ALIGN), (dict(out=A + 8), ALIGN),
    (dict(kc=A + 8), ALIGN), (dict(vc=A + 8), ALIGN), (dict(cs=A + 4), ALIGN), (dict(qs=260), ALIGN),
    (dict(ks=132), ALIGN), (dict(vs=130), ALIGN),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("over,status", BAD, ids=lambda x: str(x))
def test_refused(q8, over, status):
    assert call(q8, **over) == status


@pytest.mark.parametrize("over,status", [(dict(P=4), UNSUP), (dict(P=512), UNSUP), (dict(ksc=None), NULL),
                                         (dict(vsc=None), NULL)], ids=str)
def test_refused_by_the_8_bit_cache(over, status):
    assert call(True, **over) == status


@pytest.mark.parametrize("q8", [False, True])
def test_empty_calls_and_optional_arguments(q8):
    assert call(q8, T=0, q=None, k=None, v=None, slots=None, out=None, kc=None, vc=None) == OK
    if not torch.cuda.is_available():      # every check passed: the next thing is the device
        assert call(q8) == NODEV
        assert call(q8, rot=0, pos=None, cs=None) == NODEV
        assert call(q8, Hq=0, q=None, out=None, qs=0) == NODEV
        assert call(q8, q=A, out=A) == NODEV


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(cpsa.CpsaError, match="CUDA tensor"):
        cpsa.cpp_rope_kv_cache_write(None, x, x, None, None, slots, cache, cache, None, err)
    with pytest.raises(cpsa.CpsaError, match="inconsistent shapes"):
        cpsa.cpp_rope_kv_cache_write(None, x, x[:2], None, None, slots, cache, cache, None, err)
    with pytest.raises(cpsa.CpsaError, match="inconsistent shapes"):
        cpsa.cpp_rope_kv_cache_write(x, x, x, slots, None, slots, cache, cache, x, err)
    with pytest.raises(cpsa.CpsaError, match="inconsistent shapes"):
        cpsa.cpp_rope_kv_cache_write_q8(x, x, x, None, None, slots, cache, cache, cache, cache, None, err)
