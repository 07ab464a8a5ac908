"""AttentionStep.run refuses arguments that its step would not look at (CPU: raised before any device call)."""
import pytest
import torch

import chunked_prefill_paged_slot_gb300 as cpsa


def fused_step():
    """A step with the KV write fused, without the device memory that its constructor takes."""
    s = cpsa.AttentionStep.__new__(cpsa.AttentionStep)
    s.fused_kv_write, s.rope, s.rope_interleaved, s.q8, s.q_rot = True, None, False, False, None
    s.workspaces, s.dev_err, s.max_kv_splits = [None], None, 8
    return s


@pytest.mark.parametrize("extra,match", [
    (dict(positions=torch.zeros(1, dtype=torch.int64)), "positions go with"),
    (dict(k_scale=torch.zeros(1, dtype=torch.uint8)), "k_scale and v_scale go with"),
    (dict(v_scale=torch.zeros(1, dtype=torch.uint8)), "k_scale and v_scale go with"),
    (dict(k_scale=torch.zeros(1, dtype=torch.uint8), v_scale=torch.zeros(1, dtype=torch.uint8)),
     "k_scale and v_scale go with")], ids=["positions", "k_scale", "v_scale", "both scales"])
def test_fused_step_takes_neither_positions_nor_scales(extra, match, monkeypatch):
    """Unrotated keys would go into the cache, or a scale be passed over, without a word."""
    from chunked_prefill_paged_slot_gb300 import step
    calls = []
    monkeypatch.setattr(step._lib, "cpp_chunked_prefill_attn_write_kv", lambda *a, **k: calls.append(a))
    with pytest.raises(cpsa.CpsaError, match=match):
        fused_step().run(*[None] * 10, **extra)
    assert not calls
    fused_step().run(*[None] * 10)
    assert len(calls) == 1
