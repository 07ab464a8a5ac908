"""The package works with a torch that has no type for pairs of 4-bit floats: the 4-bit cache is plain bytes then."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
if hasattr(torch, "float4_e2m1fn_x2"):
    del torch.float4_e2m1fn_x2
import chunked_prefill_paged_slot_gb300 as cpsa
held = [torch.zeros(4, 2, 16, n, dtype=torch.uint8) for n in (32, 32, 4, 4)]
x, slots, err = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64), torch.zeros(1, dtype=torch.int32)
for call in (lambda: cpsa.cpp_rope_kv_cache_write_q4(None, x, x, None, None, slots, *held, None, err),
             lambda: cpsa.cpp_kv_cache_read_q4(*held, slots, x, x, err),
             lambda: cpsa.AttentionStep(1, 1, 2, 2, 64, device="cpu", kv_dtype=torch.float16),
             lambda: cpsa.AttentionStep(1, 1, 2, 2, 64, device="cpu", kv_dtype=None)):
    try:
        call()
    except cpsa.CpsaError as e:
        print("refused:", e)
"""


def test_import_and_refusals():
    done = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr[-2000:]
    lines = done.stdout.splitlines()
    assert len(lines) == 4 and all("CUDA tensor" in x for x in lines[:2]) and all("kv_dtype must be" in x for x in lines[2:])
