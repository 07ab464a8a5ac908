"""A missing tensor is refused as a CpsaError, by every call of the head norms and the 4-bit cache, whichever tensor it is."""
import inspect

import pytest
import torch

import chunked_prefill_paged_slot_gb300 as cpsa

APPENDS = ["cpp_norm_rope_kv_cache_write", "cpp_norm_rope_kv_cache_write_q8", "cpp_norm_rope_kv_cache_write_q4",
           "cpp_rope_kv_cache_write_q4"]
CALLS = APPENDS + ["cpp_kv_cache_read_q4", "cpp_chunked_prefill_attn_q4"]


def arguments(name, device):
    """A small call: 3 tokens, 4/2 heads of 64 columns, 4 pages of 16."""
    x = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16, device=device)
    i = lambda kind, *v: torch.tensor(v, dtype=kind, device=device)
    byte = lambda *shape: torch.zeros(*shape, dtype=torch.uint8, device=device)
    a = dict(q=x(3, 4, 64), k=x(3, 2, 64), v=x(3, 2, 64), q_weight=torch.ones(64, device=device),
             k_weight=torch.ones(64, device=device), positions=i(torch.int64, 0, 1, 2),
             cos_sin=torch.ones(8, 64, device=device), slot_mapping=i(torch.int64, 0, 1, 2), q_out=x(3, 4, 64),
             query_lens=i(torch.int32, 3), seq_lens=i(torch.int32, 3), block_table=i(torch.int32, 0).view(1, 1),
             out=x(3, 4, 64), workspace=byte(32 << 20), dev_err=i(torch.int32, 0))
    if name.endswith("_q4"):
        a |= dict(k_cache=byte(4, 2, 16, 32), v_cache=byte(4, 2, 16, 32), k_scale=byte(4, 2, 16, 4), v_scale=byte(4, 2, 16, 4))
    elif name.endswith("_q8"):
        a |= dict(k_cache=byte(4, 2, 16, 64), v_cache=byte(4, 2, 16, 64), k_scale=byte(4, 2, 1), v_scale=byte(4, 2, 1))
    else:
        a |= dict(k_cache=x(4, 2, 16, 64), v_cache=x(4, 2, 16, 64))
    return {p: a[p] for p in inspect.signature(getattr(cpsa, name)).parameters if p in a}


@pytest.mark.parametrize("name", [n for n in APPENDS if "norm" in n])
@pytest.mark.parametrize("weight", ["q_weight", "k_weight"])
def test_norm_weights_on_the_host(name, weight):
    """(Before the device of any tensor is looked at.)"""
    a = arguments(name, "cpu")
    a[weight] = None
    with pytest.raises(cpsa.CpsaError, match="k_weight, and q_weight with q"):
        getattr(cpsa, name)(**a)


@pytest.mark.parametrize("name", CALLS)
def test_any_tensor_on_the_host(name):
    for missing in arguments(name, "cpu"):
        a = arguments(name, "cpu")
        a[missing] = None
        with pytest.raises(cpsa.CpsaError):
            getattr(cpsa, name)(**a)


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_any_tensor(cuda_lib, name):
    a = arguments(name, "cuda")
    getattr(cpsa, name)(**a)
    assert cpsa.cpp_read_device_error(a["dev_err"]) == 0
    for missing in a:
        with pytest.raises(cpsa.CpsaError):
            getattr(cpsa, name)(**(a | {missing: None}))
