"""AttentionStep as its constructor leaves it, on the CPU: what its run calls and refuses, for every kind of step."""
import pytest
import torch

import chunked_prefill_paged_slot_gb300 as cpsa
from chunked_prefill_paged_slot_gb300 import step

W = torch.ones(64)
ROPE = torch.ones(8, 64)
KINDS = {"bf16": {}, "fused": dict(fused_kv_write=True), "8 bit": dict(kv_dtype=torch.float8_e4m3fn),
         "4 bit": dict(kv_dtype=torch.float4_e2m1fn_x2), "bf16 rope": dict(rope=ROPE),
         "4 bit rope": dict(kv_dtype=torch.float4_e2m1fn_x2, rope=ROPE), "bf16 norm": dict(q_norm=W, k_norm=W),
         "8 bit norm rope": dict(kv_dtype=torch.float8_e4m3fn, q_norm=W, k_norm=W, rope=ROPE),
         "4 bit norm rope": dict(kv_dtype=torch.float4_e2m1fn_x2, q_norm=W, k_norm=W, rope=ROPE)}


@pytest.fixture
def calls(monkeypatch):
    """Constructors without a GPU (no pinned memory), and the names of the library's calls in place of the calls."""
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, pin_memory=False, **k: zeros(*a, **k))
    names = []
    for name in [n for n in dir(step._lib) if n.startswith("cpp_") and n != "cpp_attn_workspace_bytes"]:
        monkeypatch.setattr(step._lib, name, lambda *a, _name=name, **k: names.append(_name))
    return names


def build(kind):
    return cpsa.AttentionStep(1, 3, 4, 2, 64, device="cpu", **KINDS[kind])


def run(s, **kw):
    s.run(torch.zeros(3, 4, 64), *[None] * 9, **kw)


def extras(kind):
    scale = torch.zeros(1, dtype=torch.uint8)
    return (dict(positions=torch.zeros(3, dtype=torch.int64)) if "rope" in kind else {}) | (
        dict(k_scale=scale, v_scale=scale) if "bit" in kind else {})


@pytest.mark.parametrize("kind", KINDS)
def test_run_makes_its_calls(calls, kind):
    run(build(kind), **extras(kind))
    bits = {"8": "_q8", "4": "_q4"}.get(kind[0], "")
    if kind == "fused":
        assert calls == ["cpp_chunked_prefill_attn_write_kv"]
        return
    write = "cpp_norm_rope_kv_cache_write" if "norm" in kind else "cpp_rope_kv_cache_write" if kind != "bf16" else "cpp_kv_cache_write"
    assert calls == [write + bits, "cpp_chunked_prefill_attn" + bits]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("other", ["positions", "k_scale", "v_scale"])
def test_run_refuses_what_its_step_would_not_look_at(calls, kind, other):
    kw = extras(kind)
    if other in kw:
        del kw[other]
    else:
        kw[other] = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(cpsa.CpsaError, match="go with"):
        run(build(kind), **kw)
    assert not calls


@pytest.mark.parametrize("kind", KINDS)
def test_nothing_of_a_step_is_left_to_its_class(calls, kind):
    """Every attribute that run may look at is the instance's own."""
    s = build(kind)
    assert not [n for n, v in vars(cpsa.AttentionStep).items() if not n.startswith("_") and not callable(v)]
    assert {"q8", "q4", "norm", "norm_eps", "rope", "q_rot", "fused_kv_write"} <= set(vars(s))
