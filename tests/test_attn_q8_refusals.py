"""cpp_chunked_prefill_attn_q8 refuses what it cannot do before anything is launched (CPU: no device is touched)."""
import pytest
import torch

import chunked_prefill_paged_slot_gb300 as cpsa

A = 0x10000          # an aligned address that is never read


def call(**over):
    a = dict(q=A, kc=A, vc=A, ks=A, vs=A, ql=A, sl=A, bt=A, B=2, T=5, M=4, Hq=4, Hkv=2, d=64, P=16, pages=8, scale=0.0,
             splits=8, out=A, ws=A, wsb=1 << 30, err=A, stream=None)
    assert set(over) <= set(a), over
    a.update(over)
    return cpsa.load().cpp_chunked_prefill_attn_q8(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(ks=None), -1), (dict(vs=None), -1), (dict(q=None), -1), (dict(kc=None), -1), (dict(vc=None), -1),
    (dict(ql=None), -1), (dict(sl=None), -1), (dict(bt=None), -1), (dict(out=None), -1), (dict(ws=None), -1),
    (dict(err=None), -1), (dict(B=-1), -2), (dict(T=-1), -2), (dict(B=0), -2), (dict(M=-1), -2), (dict(pages=-1), -2),
    (dict(pages=1 << 40), -2), (dict(splits=0), -2), (dict(splits=33), -2), (dict(q=A + 8), -3), (dict(kc=A + 8), -3),
    (dict(vc=A + 8), -3), (dict(out=A + 2), -3), (dict(ws=A + 4), -3), (dict(d=96), -4), (dict(P=4), -4), (dict(P=24), -4),
    (dict(P=512), -4), (dict(Hq=5), -4), (dict(Hq=34), -4), (dict(wsb=100), -5)], ids=str)
def test_refused(over, status):
    assert call(**over) == status


def test_empty_call():
    assert call(T=0, B=0, q=None, ks=None, vs=None) == 0
    if not torch.cuda.is_available():
        assert call() == -7


def test_binding_refuses_wrong_types_and_shapes():
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(cpsa.CpsaError, match="k_cache must be"):
        c = torch.zeros(2, 2, 16, 64, dtype=torch.uint8)
        i = torch.zeros(1, dtype=torch.int32)
        cpsa.cpp_chunked_prefill_attn_q8(q, c, c, c, c, i, i, i.view(1, 1), q, c.view(-1), i)
