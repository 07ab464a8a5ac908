"""Performance cases of head norms with the rotary KV append, and of the 4-bit paged KV cache.

Four operators of one serving step and of what moves its cache about:

  norm_rope  cpp_norm_rope_kv_cache_write: RMS norm of every q and k head, rotation by
             position, q written out, k and v appended to the bf16 paged cache
  q4_append  cpp_rope_kv_cache_write_q4: rotate and append into a 4-bit cache, then
             cpp_kv_cache_read_q4 of the same slots (so that what is held in 4 bits
             comes back as the values it stands for)
  q4_read    cpp_kv_cache_read_q4: rows of the 4-bit cache, gathered by slot, as bf16
  attn_q4    cpp_chunked_prefill_attn_q4: causal attention of prefill chunks and decode
             rows over the 4-bit cache

`run` computes each in its plain form (elementary torch operations in fp32), or,
with `own` set, through the library's entry points. `exact` is the same from the
definitions in 64 bits.

The definitions:
  norm       y_c = x_c / sqrt(mean_c x_c^2 + eps) * w_c over the head's columns c
  rotation   pair (a, b) of a head at angle t: (a cos t - b sin t, b cos t + a sin t);
             pair i is (x[i], x[i + rot/2]), or (x[2i], x[2i + 1]) when interleaved;
             columns from rot on pass through. cos and sin come from a table.
  4 bits     value = code * scale, a scale for every 16 columns of a place and head.
             Codes: sign and 0, 0.5, 1, 1.5, 2, 3, 4, 6 (e2m1), two to a byte, the even
             column in the low half. Scales: 5 bits of exponent and 3 of mantissa, no
             sign: the upper byte of the f16 number's 15 bits behind its sign, so from
             2^-17 on; all ones are NaN. scale = amax / 6 to the nearest such number (ties to
             even), at least 2^-17, at most 10240; codes are x / scale to the nearest (ties
             to even), at most 6 in magnitude. A NaN or infinity among the 16 makes them NaN.
  attention  out = sum_j softmax_j(q . k_j / sqrt(d)) v_j over the keys 0 .. h + i of
             new token i of a request with h cached tokens before it.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

EPS = 1e-6
GROUP = 16                # columns that share a scale
NAN_SCALE = 255           # what places of the 4-bit cache behind a sequence hold here


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    llama = dict(hq=32, hkv=8, d=128)
    small = dict(hq=14, hkv=2, d=64)
    return [
        # one user's next token: launch latency
        dict(name="norm_rope_1_token", op="norm_rope", decode=1, prompts=0, qlen=0, pad=0, page=16, rot=128, inter=False, **llama),
        # a token budget of 2048: 1536 decode rows and a chunk of 512
        dict(name="norm_rope_budget2048", op="norm_rope", decode=1536, prompts=1, qlen=512, pad=0, page=16, rot=128, inter=False, **llama),
        # ragged prompts of a small grouped model, partial interleaved rotation
        dict(name="norm_rope_ragged_d64", op="norm_rope", decode=37, prompts=7, qlen=1187, pad=11, page=32, rot=32, inter=True, **small),
        # a decode step of 125 rows padded to 128
        dict(name="q4_append_decode128", op="q4_append", decode=125, prompts=0, qlen=0, pad=3, page=16, rot=128, inter=False, **llama),
        # a whole 32768-token prompt in one call
        dict(name="q4_append_prompt32768", op="q4_append", decode=0, prompts=1, qlen=32768, pad=0, page=128, rot=128, inter=False, **llama),
        # a short prefix of a small model, odd length
        dict(name="q4_read_777_d64", op="q4_read", decode=0, prompts=1, qlen=777, pad=0, page=32, **small),
        # prefixes of 8192 tokens handed on to another cache
        dict(name="q4_read_prefixes", op="q4_read", decode=0, prompts=4, qlen=8192, pad=5, page=16, **llama),
        # one user's next token over a short context: launch latency
        dict(name="attn_q4_1_row", op="attn_q4", decode=1, lo=777, hi=777, prompts=0, qlen=0, hist=0, page=16, **llama),
        # decode rows of the mixed workload's contexts: the cache's bandwidth
        dict(name="attn_q4_decode384", op="attn_q4", decode=384, lo=1024, hi=8192, prompts=0, qlen=0, hist=0, page=16, **llama),
        # the last chunk of a 32768-token prompt: the tensor cores' rate
        dict(name="attn_q4_chunk_h32256", op="attn_q4", decode=0, lo=1, hi=1, prompts=1, qlen=512, hist=32256, page=128, **llama),
        # decode rows and a chunk in one step
        dict(name="attn_q4_mixed", op="attn_q4", decode=96, lo=1024, hi=8192, prompts=1, qlen=512, hist=8192, page=16, **llama),
        # fresh ragged prompts of a small model, one q head at a time (7 q heads per kv head)
        dict(name="attn_q4_ragged_d64", op="attn_q4", decode=5, lo=60, hi=900, prompts=6, qlen=1187, hist=0, page=32, **small),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv, d = rng.choice([(32, 8, 128), (32, 8, 128), (16, 4, 128), (8, 1, 128), (6, 3, 128), (14, 2, 64), (4, 4, 64)])
    page = rng.choice([8, 16, 16, 32, 64, 128, 256])
    heads = dict(hq=hq, hkv=hkv, d=d, page=page)
    op = rng.choice(["norm_rope", "q4_append", "q4_read", "attn_q4", "attn_q4"])
    kind = rng.choice(["decode", "chunk", "mixed"])
    decode = _log(rng, 1, 300) if kind != "chunk" else 0
    prompts = rng.randint(1, 4) if kind != "decode" else 0
    if op == "attn_q4":
        lo = _log(rng, 1, 3000)
        return dict(op=op, decode=decode, lo=lo, hi=lo + _log(rng, 1, 4000), prompts=prompts,
                    qlen=_log(rng, 2, 1200) if prompts else 0, hist=rng.choice([0, _log(rng, 1, 12000)]) if prompts else 0, **heads)
    case = dict(op=op, decode=decode * rng.randint(1, 5), prompts=prompts, qlen=_log(rng, 2, 6000) if prompts else 0,
                pad=rng.choice([0, 0, 5]), **heads)
    if op != "q4_read":
        case |= dict(rot=rng.choice([d, d, d // 2, 16]), inter=rng.random() < 0.3)
    return case


def work(case):
    lens = _lengths(case, 0)
    tokens = sum(q for _, q in lens)
    hq, hkv, d, op = case["hq"], case["hkv"], case["d"], case["op"]
    held = 2 * hkv * (d // 2 + d // GROUP)                          # a place of the 4-bit cache, k and v
    if op == "attn_q4":
        keys = sum(h + q for h, q in lens)
        pairs = sum(q * h + q * (q + 1) // 2 for h, q in lens)
        return {"bytes": keys * held + 4 * tokens * hq * d + 4 * keys // case["page"], "flops": 4 * d * hq * pairs}
    if op == "q4_read":
        return {"bytes": tokens * (held + 4 * hkv * d + 8), "flops": tokens * 2 * hkv * d}
    moved = tokens * d * (4 * hq + 4 * hkv)                          # q in and out, k and v in
    moved += tokens * (16 + 4 * case["rot"])                         # position, slot, the table's row
    if op == "norm_rope":
        return {"bytes": moved + tokens * d * 4 * hkv + 8 * d, "flops": tokens * (hq + hkv) * (4 * d + 3 * case["rot"])}
    return {"bytes": moved + tokens * (held + 4 * hkv * d), "flops": tokens * ((hq + hkv) * case["rot"] * 3 + 6 * hkv * d)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(case, seed):
    """(tokens cached before, new tokens) of every request: decode rows first."""
    r = np.random.RandomState(seed % (1 << 31))
    if case["op"] == "attn_q4":
        lens = [(int(c) - 1, 1) for c in r.randint(case["lo"], case["hi"] + 1, case["decode"])]
    else:
        lens = [(int(c), 1) for c in r.randint(0, 8192, case["decode"])]
    r = np.random.RandomState(case["qlen"])      # the same prompts for every seed: their outputs have one shape
    for i in range(case["prompts"]):
        q = case["qlen"] if i == 0 else max(2, case["qlen"] - int(r.randint(0, case["qlen"] // 2 + 1)))
        hist = case["hist"] if case["op"] == "attn_q4" else (0 if i % 2 == 0 else int(r.randint(1, 300)))
        lens.append((hist, q))
    return lens


def _code_pairs():
    """Bytes of two codes, each the code of a normal number under the scale of the largest of 16: one for each of 2^16 places."""
    edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    share = torch.special.ndtr(edge / 3.0)                          # 6 stands for two standard deviations
    u = (torch.arange(256, dtype=torch.float64) + 0.5) / 256
    code = (2 * (u - 0.5).abs() + 1).div(2)[:, None].gt(share).sum(1) + 8 * (u < 0.5)
    return (code[:, None] + 16 * code[None, :]).flatten().to(torch.uint8).cuda()


def _held(pages, case, gen):
    """Codes and scales of normal data."""
    hkv, page, d = case["hkv"], case["page"], case["d"]
    place = torch.randint(0, 65536, (pages, hkv, page, d // 2), generator=gen, device="cuda", dtype=torch.int32)
    scale = torch.randint(101, 111, (pages, hkv, page, d // GROUP), generator=gen, device="cuda", dtype=torch.uint8)
    return _code_pairs()[place], scale


def prepare(case, seed):
    lens = _lengths(case, seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    r = np.random.RandomState((int(seed) + 1) % (1 << 31))
    hq, hkv, d, page, op = case["hq"], case["hkv"], case["d"], case["page"], case["op"]
    if op == "attn_q4":
        need = [(h + q + page - 1) // page for h, q in lens]
        pages = sum(need)
        order = r.permutation(pages)
        table = np.full((len(lens), max(need)), -1, np.int32)
        ends = np.cumsum(need)
        for i, n in enumerate(need):
            table[i, :n] = order[ends[i] - n:ends[i]]
        tokens = sum(q for _, q in lens)
        s = dict(case=case, lens=lens, pages=pages,
                 q=torch.randn((tokens, hq, d), generator=gen, device="cuda").to(torch.bfloat16),
                 out=torch.zeros((tokens, hq, d), device="cuda", dtype=torch.bfloat16),
                 query_lens=torch.tensor([q for _, q in lens], dtype=torch.int32, device="cuda"),
                 seq_lens=torch.tensor([h + q for h, q in lens], dtype=torch.int32, device="cuda"),
                 block_table=torch.from_numpy(table).cuda(),
                 dev_err=torch.zeros(1, dtype=torch.int32, device="cuda"))
        # places behind a sequence hold NaN
        last = np.array([table[i, n - 1] for i, n in enumerate(need)])
        used = np.array([h + q - (n - 1) * page for (h, q), n in zip(lens, need)])
        at, row = np.nonzero(np.arange(page)[None, :] >= used[:, None])
        at, row = torch.from_numpy(last[at]).cuda(), torch.from_numpy(row).cuda()
        for name in ("k", "v"):
            s[name + "_cache"], s[name + "_scale"] = _held(pages, case, gen)
            s[name + "_scale"][at, :, row] = NAN_SCALE
        return s
    # every request has the pages that its new tokens touch
    first = [h // page for h, _ in lens]
    need = [(h + q - 1) // page - f + 1 for (h, q), f in zip(lens, first)]
    pages = sum(need) + 7
    order = r.permutation(pages).astype(np.int64)
    slots, places, at = [], [], 0
    for (h, q), f, n in zip(lens, first, need):
        p = np.arange(h, h + q, dtype=np.int64)
        slots.append(order[at + p // page - f] * page + p % page)
        places.append(p)
        at += n
    pad = np.full(case["pad"], -1, np.int64)
    slots, places = np.concatenate(slots + [pad]), np.concatenate(places + [pad])
    tokens = len(slots)
    s = dict(case=case, pages=pages, slot_mapping=torch.from_numpy(slots).cuda(),
             dev_err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if op == "norm_rope":
        for name in ("k_cache", "v_cache"):
            s[name] = torch.randn((pages, hkv, page, d), generator=gen, device="cuda").to(torch.bfloat16)
    else:
        for name in ("k", "v"):
            s[name + "_cache"], s[name + "_scale"] = _held(pages, case, gen)
            s[name + "_back"] = torch.zeros((tokens, hkv, d), device="cuda", dtype=torch.bfloat16)
    if op == "q4_read":
        return s
    # one projection's output holds q, k and v of a token side by side
    qkv = torch.randn((tokens, (hq + 2 * hkv) * d), generator=gen, device="cuda")
    qkv[:, hq * d:(hq + hkv) * d] *= torch.exp(0.5 * torch.randn(hkv * d, generator=gen, device="cuda"))
    qkv = qkv.to(torch.bfloat16)
    rot, top = case["rot"], int(places.max()) + 1
    angle = torch.arange(top, dtype=torch.float64, device="cuda")[:, None] * (
        10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot))
    s |= dict(qkv=qkv, q=qkv[:, :hq * d].unflatten(1, (hq, d)), k=qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
              v=qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)),
              cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(), positions=torch.from_numpy(places).cuda(),
              q_out=torch.zeros((tokens, hq, d), device="cuda", dtype=torch.bfloat16))
    if op == "norm_rope":
        for name in ("q_weight", "k_weight"):
            s[name] = 1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        _own(s, op)
    elif op == "attn_q4":
        _plain_attention(s)
    elif op == "q4_read":
        _plain_read(s)
    else:
        _plain_append(s)
        if op == "q4_append":
            _plain_read(s)
    if op == "attn_q4":
        return s["out"]
    if op == "norm_rope":
        return {"q_out": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    back = {"k": s["k_back"], "v": s["v_back"]}
    return back if op == "q4_read" else back | {"q_out": s["q_out"]}


def _own(s, op):
    import chunked_prefill_paged_slot_gb300 as cpsa
    if op == "norm_rope":
        cpsa.cpp_norm_rope_kv_cache_write(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["positions"],
                                          s["cos_sin"], s["slot_mapping"], s["k_cache"], s["v_cache"], s["q_out"],
                                          s["dev_err"], eps=EPS, interleaved=s["case"]["inter"])
        return
    caches = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if op == "attn_q4":
        if "workspace" not in s:      # a user's program keeps it from step to step
            c = s["case"]
            size = cpsa.cpp_attn_workspace_bytes(len(s["lens"]), s["q"].shape[0], c["hq"], c["hkv"], c["d"], 8)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        cpsa.cpp_chunked_prefill_attn_q4(s["q"], *caches, s["query_lens"], s["seq_lens"], s["block_table"], s["out"],
                                         s["workspace"], s["dev_err"])
        return
    if op == "q4_append":
        cpsa.cpp_rope_kv_cache_write_q4(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slot_mapping"], *caches,
                                        s["q_out"], s["dev_err"], interleaved=s["case"]["inter"])
    cpsa.cpp_kv_cache_read_q4(*caches, s["slot_mapping"], s["k_back"], s["v_back"], s["dev_err"])


# ---------------------------------------------------------------------------
# the plain forms, in fp32
# ---------------------------------------------------------------------------
def _rotate(x, cos, sin, rot, inter):
    """x [n, heads, d] fp32; cos, sin [n, 1, rot / 2]."""
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    if inter:
        y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ra, rb
    return y


def _plain_append(s):
    c = s["case"]
    rot, page = c["rot"], c["page"]
    live = s["positions"] >= 0
    table = s["cos_sin"][s["positions"][live]][:, None, :]
    cos, sin = table[..., :rot // 2], table[..., rot // 2:]
    q, k, v, slot = s["q"][live].float(), s["k"][live].float(), s["v"][live].float(), s["slot_mapping"][live]
    if c["op"] == "norm_rope":
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["q_weight"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["k_weight"]
    s["q_out"][live] = _rotate(q, cos, sin, rot, c["inter"]).to(torch.bfloat16)
    k = _rotate(k, cos, sin, rot, c["inter"])
    k, v, slot = k[slot >= 0], v[slot >= 0], slot[slot >= 0]
    at, off = slot // page, slot % page
    if c["op"] == "norm_rope":
        s["k_cache"][at, :, off] = k.to(torch.bfloat16)
        s["v_cache"][at, :, off] = v.to(torch.bfloat16)
    else:
        s["k_cache"][at, :, off], s["k_scale"][at, :, off] = _quantised(k)
        s["v_cache"][at, :, off], s["v_scale"][at, :, off] = _quantised(v)


def _quantised(x):
    """x [n, heads, d] fp32 as (bytes of two codes, scale bytes)."""
    x = x.unflatten(-1, (-1, GROUP))
    want = x.abs().amax(-1)
    want = want / torch.full_like(want, 6.0)      # a division: by a number torch multiplies by its reciprocal, and ties are no ties then
    bits = want.view(torch.int32)
    scale = torch.where(want < 2.0 ** -14, torch.round(want * 2.0 ** 17) * 2.0 ** -17,
                        (bits + 0x7FFFF + ((bits >> 20) & 1) >> 20 << 20).view(torch.float32)).clamp(2.0 ** -17, 10240.0)
    y = x / scale[..., None]
    size = y.abs()
    size = torch.where(size < 2, torch.round(size * 2) / 2, torch.where(size < 4, torch.round(size), torch.round(size / 2) * 2)).clamp(max=6.0)
    code = torch.where(size <= 2, size * 2, torch.where(size <= 4, size + 2, size + 1)) + 8.0 * (y < 0)
    fine = torch.isfinite(want)
    byte = torch.where(fine, (scale.to(torch.float16).view(torch.int16) >> 7).int(), NAN_SCALE).to(torch.uint8)
    code = torch.where(fine[..., None], code, 7.0).to(torch.uint8).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], byte


def _code_table():
    """The two values of every byte of codes, [256, 2]."""
    one = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    one = torch.cat([one, -one])
    return torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)


def _values(codes, scale):
    """What codes [..., d / 2] under scale [..., d / 16] stand for, [..., d] fp32."""
    x = _code_table()[codes.int()].flatten(-2).unflatten(-1, (-1, GROUP))
    return (x * (scale.short() << 7).view(torch.float16).float()[..., None]).flatten(-2)


def _plain_read(s):
    page = s["case"]["page"]
    live = s["slot_mapping"] >= 0
    slot = s["slot_mapping"][live]
    at, off = slot // page, slot % page
    for name in ("k", "v"):
        s[name + "_back"][live] = _values(s[name + "_cache"][at, :, off], s[name + "_scale"][at, :, off]).to(torch.bfloat16)


def _plain_attention(s):
    lens = s["lens"]
    decode = [i for i, (_, q) in enumerate(lens) if q == 1]
    prompts = [i for i, (_, q) in enumerate(lens) if q > 1]
    if decode:
        _plain_requests(s, decode)
    if prompts:
        _plain_requests(s, prompts)


def _plain_requests(s, which):
    """The rows of the requests `which`, padded to the longest of them."""
    c, lens = s["case"], s["lens"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    start = np.cumsum([0] + [q for _, q in lens])
    hist = torch.tensor([lens[i][0] for i in which], device="cuda")
    qlen = torch.tensor([lens[i][1] for i in which], device="cuda")
    first = torch.tensor([int(start[i]) for i in which], device="cuda")
    most_q, most_k = max(lens[i][1] for i in which), max(sum(lens[i]) for i in which)
    n, keys = len(which), -(-most_k // page) * page
    at = s["block_table"][torch.tensor(which, device="cuda"), :keys // page].clamp(min=0).long()

    def values(name):
        x = _values(s[name + "_cache"][at], s[name + "_scale"][at])
        return x.transpose(1, 2).reshape(n, hkv, keys, d)

    i = torch.arange(most_q, device="cuda")
    row = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(n, most_q, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    j = torch.arange(keys, device="cuda")
    seen = (j <= (hist[:, None] + i)[..., None]) & (j < (hist + qlen)[:, None, None])       # [n, most_q, keys]
    score = (q @ values("k").transpose(2, 3)).view(n, hkv, hq // hkv, most_q, keys) / math.sqrt(d)
    score.masked_fill_(~seen[:, None, None], -math.inf)
    score -= score.amax(-1, keepdim=True)
    p = score.exp_()
    total = p.sum(-1)
    v = values("v")
    v.masked_fill_((j >= (hist + qlen)[:, None])[:, None, :, None], 0.0)
    out = (p.view(n, hkv, -1, keys) @ v).view(n, hkv, hq // hkv, most_q, d) / total[..., None]
    out = out.permute(0, 3, 1, 2, 4).reshape(n, most_q, hq, d)
    real = i < qlen[:, None]
    s["out"][row[real]] = out[real].to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attn_q4":
        return _exact_attention(s)
    slot = s["slot_mapping"]
    there = (slot >= 0).nonzero()[:, 0]
    at, off = slot[there] // case["page"], slot[there] % case["page"]
    if op == "q4_read":
        got = {}
        for name in ("k", "v"):
            x = s[name + "_back"].double()
            x[there] = _exact_held(s[name + "_cache"][at, :, off], s[name + "_scale"][at, :, off])
            got[name] = x
        return got
    rot = case["rot"]
    # the rotation as a complex product
    place = s["positions"].clamp(min=0)
    turn = torch.complex(s["cos_sin"][place, :rot // 2].double(), s["cos_sin"][place, rot // 2:].double())[:, None]

    def turned(x):
        pair = x[..., :rot].unflatten(-1, (rot // 2, 2) if case["inter"] else (2, rot // 2))
        if not case["inter"]:
            pair = pair.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z if case["inter"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., rot:]], -1)

    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    if op == "norm_rope":
        d = case["d"]
        q = q * (d / (torch.linalg.vector_norm(q, dim=-1, keepdim=True) ** 2 + d * EPS)).sqrt() * s["q_weight"].double()
        k = k * (d / (torch.linalg.vector_norm(k, dim=-1, keepdim=True) ** 2 + d * EPS)).sqrt() * s["k_weight"].double()
    q_out = s["q_out"].double()
    q_out[s["positions"] >= 0] = turned(q)[s["positions"] >= 0]
    got = {"q_out": q_out}
    for name, x in (("k", turned(k)), ("v", v)):
        if op == "norm_rope":
            held = s[name + "_cache"].double()
            held[at, :, off] = x[there]
            got[name + "_cache"] = held
        else:
            back = s[name + "_back"].double()
            back[there] = _exact_rounded(x[there])
            got[name] = back
    return got


def _exact_held(codes, scale):
    table = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), dtype=torch.float64, device="cuda")
    x = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    e, m = (scale >> 3).double(), (scale & 7).double()
    f = torch.where(e == 0, m * 2.0 ** -17, (8 + m) * torch.exp2(e - 18))
    f = torch.where(e == 31, torch.where(m == 0, math.inf, math.nan), f)
    return x * f.repeat_interleave(GROUP, -1)


def _exact_rounded(x):
    """x [n, heads, d] in 64 bits as the 4-bit cache holds it: the nearest of each table's numbers by bisection."""
    x = x.unflatten(-1, (-1, GROUP))
    scales = torch.cat([torch.arange(1, 8, dtype=torch.float64) * 2.0 ** -17,
                        ((8 + torch.arange(8, dtype=torch.float64)) * torch.exp2(torch.arange(-17.0, 11.0, dtype=torch.float64))[:, None]).flatten()])
    scales = scales[scales <= 10240.0].cuda()
    f = _nearest(x.abs().amax(-1) / 6.0, scales, 1)
    return (torch.sign(x) * _nearest(x.abs() / f[..., None], torch.tensor(_E2M1, dtype=torch.float64, device="cuda"), 0) * f[..., None]).flatten(-2)


def _nearest(x, table, first):
    """The number of `table` (ascending; its first is number `first` of the format) nearest to x, ties to the even one."""
    half = (table[1:] + table[:-1]) / 2
    below = torch.searchsorted(half, x.contiguous())                         # a tie goes down
    above = torch.searchsorted(half, x.contiguous(), right=True)             # a tie goes up
    return table[torch.where((below + first) % 2 == 0, below, above)]


def _exact_attention(s):
    c = s["case"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    out, at = [], 0
    for r, (h, q) in enumerate(s["lens"]):
        n = h + q
        pages = s["block_table"][r, :-(-n // page)].long()
        k, v = (_exact_held(s[x + "_cache"][pages], s[x + "_scale"][pages]).transpose(1, 2).reshape(-1, hkv, d)[:n]
                .transpose(0, 1).repeat_interleave(hq // hkv, 0) for x in ("k", "v"))
        z = torch.bmm(s["q"][at:at + q].double().transpose(0, 1), k.transpose(1, 2)) / math.sqrt(d)
        if q > 1:
            hidden = torch.ones((q, n), dtype=torch.bool, device="cuda").triu(h + 1)
            z.masked_fill_(hidden, -math.inf)
        out.append(torch.bmm(torch.softmax(z, -1), v).transpose(0, 1))
        at += q
    return torch.cat(out)
