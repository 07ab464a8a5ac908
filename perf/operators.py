"""Performance cases of the rotary KV append and of the 8-bit paged KV cache.

Three operators of one serving step, in the order in which a layer calls them:

  rope      cpp_rope_kv_cache_write: rotate the new tokens' q and k by their
            positions, write q_out, append k and v to the bf16 paged cache
  rope_q8   cpp_rope_kv_cache_write_q8: the same into a cache of e4m3 bytes with
            one power-of-two scale per (page, kv head, block of min(16, page)
            tokens)
  attn_q8   cpp_chunked_prefill_attn_q8: causal attention of prefill chunks and
            decode rows over that 8-bit cache

`run` computes each in its plain form (elementary torch operations in fp32), or,
with `own` set, through the library's entry points. `exact` is the same from the
definitions in 64 bits.

The definitions:
  rotation   pair (a, b) of a head at angle t: (a cos t - b sin t, b cos t + a sin t);
             pair i is (x[i], x[i + rot/2]), or (x[2i], x[2i + 1]) when interleaved;
             columns from rot on pass through. cos and sin come from a table.
  8 bits     value = e4m3 byte * 2^(scale byte - 127). For the tokens that a call
             puts into a block, need = the smallest x with amax <= 448 * 2^x over
             their finite values, within [-117, 119]. If they include the block's
             first place, the block starts over with x = need; else x = max(need,
             the block's x), and where that is larger than before, the block's other
             bytes are rounded to the new scale. Bytes are rounded to nearest even,
             saturating at 448; infinities and NaN become NaN.
  attention  out = sum_j softmax_j(q . k_j / sqrt(d)) v_j over the keys 0 .. h + i of
             new token i of a request with h cached tokens before it.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

NEW_PAGE_BYTE = 0x7F      # NaN: what unwritten places of the 8-bit cache hold here


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    llama = dict(hq=32, hkv=8, d=128)
    return [
        # one user's next token: launch latency
        dict(name="rope_1_token", op="rope", decode=1, prompts=0, qlen=0, pad=0, page=16, rot=128, inter=False, **llama),
        # a token budget of 2048: 1536 decode rows and a chunk of 512
        dict(name="rope_budget2048", op="rope", decode=1536, prompts=1, qlen=512, pad=0, page=16, rot=128, inter=False, **llama),
        # ragged prompts of a small grouped model, partial interleaved rotation
        dict(name="rope_ragged_d64", op="rope", decode=37, prompts=7, qlen=1187, pad=11, page=32, rot=32, inter=True, hq=14, hkv=2, d=64),
        # a decode step of 125 rows padded to 128
        dict(name="rope_q8_decode128", op="rope_q8", decode=125, prompts=0, qlen=0, pad=3, page=16, rot=128, inter=False, **llama),
        dict(name="rope_q8_budget2048", op="rope_q8", decode=1536, prompts=1, qlen=512, pad=0, page=16, rot=128, inter=False, **llama),
        # a whole 32768-token prompt in one call
        dict(name="rope_q8_prompt32768", op="rope_q8", decode=0, prompts=1, qlen=32768, pad=0, page=128, rot=128, inter=False, **llama),
        # one user's next token over a short context: launch latency
        dict(name="attn_q8_1_row", op="attn_q8", decode=1, lo=777, hi=777, prompts=0, qlen=0, hist=0, page=16, **llama),
        # the decode rows of the micro-batch workload
        dict(name="attn_q8_decode128", op="attn_q8", decode=128, lo=2600, hi=5200, prompts=0, qlen=0, hist=0, page=16, **llama),
        # decode rows of the mixed workload's contexts: the cache's bandwidth
        dict(name="attn_q8_decode384", op="attn_q8", decode=384, lo=1024, hi=8192, prompts=0, qlen=0, hist=0, page=16, **llama),
        # the last chunk of a 32768-token prompt: the tensor cores' rate
        dict(name="attn_q8_chunk_h32256", op="attn_q8", decode=0, lo=1, hi=1, prompts=1, qlen=512, hist=32256, page=128, **llama),
        # decode rows and a chunk in one step
        dict(name="attn_q8_mixed", op="attn_q8", decode=96, lo=1024, hi=8192, prompts=1, qlen=512, hist=8192, page=16, **llama),
        # fresh ragged prompts of a small model, one q head at a time (7 q heads per kv head)
        dict(name="attn_q8_ragged_d64", op="attn_q8", decode=5, lo=60, hi=900, prompts=6, qlen=1187, hist=0, page=32, hq=14, hkv=2, d=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv, d = rng.choice([(32, 8, 128), (32, 8, 128), (16, 4, 128), (8, 1, 128), (6, 3, 128), (14, 2, 64), (4, 4, 64)])
    page = rng.choice([8, 16, 16, 32, 64, 128, 256])
    heads = dict(hq=hq, hkv=hkv, d=d, page=page)
    op = rng.choice(["rope", "rope_q8", "attn_q8", "attn_q8"])
    kind = rng.choice(["decode", "chunk", "mixed"])
    decode = _log(rng, 1, 300) if kind != "chunk" else 0
    prompts = rng.randint(1, 4) if kind != "decode" else 0
    if op != "attn_q8":
        return dict(op=op, decode=decode * rng.randint(1, 5), prompts=prompts, qlen=_log(rng, 2, 6000) if prompts else 0,
                    pad=rng.choice([0, 0, 5]), rot=rng.choice([d, d, d // 2, 16]), inter=rng.random() < 0.3, **heads)
    lo = _log(rng, 1, 3000)
    return dict(op=op, decode=decode, lo=lo, hi=lo + _log(rng, 1, 4000), prompts=prompts,
                qlen=_log(rng, 2, 1200) if prompts else 0, hist=rng.choice([0, _log(rng, 1, 12000)]) if prompts else 0, **heads)


def work(case):
    lens = _lengths(case, 0)
    tokens = sum(q for _, q in lens)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] != "attn_q8":
        out = 2 if case["op"] == "rope" else 1
        moved = tokens * d * (4 * hq + 2 * hkv * (2 + out))          # q in and out, k and v in and out
        moved += tokens * (16 + 4 * case["rot"])                     # position, slot, the table's row
        if case["op"] == "rope_q8":
            blocks = sum((h + q - 1) // _sb(case) - h // _sb(case) + 1 for h, q in lens)
            moved += blocks * hkv * 4                                # scales read and written
        return {"bytes": moved, "flops": tokens * (hq + hkv) * case["rot"] * 3}
    keys = sum(h + q for h, q in lens)
    pairs = sum(q * h + q * (q + 1) // 2 for h, q in lens)
    return {"bytes": 2 * keys * hkv * d + 2 * keys * hkv // _sb(case) + 4 * tokens * hq * d + 4 * keys // case["page"],
            "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _sb(case):
    return min(16, case["page"])


def _lengths(case, seed):
    """(tokens cached before, new tokens) of every request: decode rows first."""
    r = np.random.RandomState(seed % (1 << 31))
    if case["op"] == "attn_q8":
        lens = [(int(c) - 1, 1) for c in r.randint(case["lo"], case["hi"] + 1, case["decode"])]
    else:
        lens = [(int(c), 1) for c in r.randint(0, 8192, case["decode"])]
    r = np.random.RandomState(case["qlen"])      # the same prompts for every seed: their outputs have one shape
    for i in range(case["prompts"]):
        q = case["qlen"] if i == 0 else max(2, case["qlen"] - int(r.randint(0, case["qlen"] // 2 + 1)))
        hist = case["hist"] if case["op"] == "attn_q8" else (0 if i % 2 == 0 else int(r.randint(1, 300)))
        lens.append((hist, q))
    return lens


def _scales(shape, gen):
    """Scale bytes of normal data: 2^-7 mostly, a step below or above for some blocks."""
    u = torch.rand(shape, generator=gen, device="cuda")
    return (120 - (u < 0.1).to(torch.uint8) + (u > 0.8).to(torch.uint8)).to(torch.uint8)


def _raw(shape, gen):
    """e4m3 bytes of normal data under such scales."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return x.mul_(110.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)


def prepare(case, seed):
    lens = _lengths(case, seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    r = np.random.RandomState((int(seed) + 1) % (1 << 31))
    hq, hkv, d, page, sb = case["hq"], case["hkv"], case["d"], case["page"], _sb(case)
    if case["op"] == "attn_q8":
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
        # places behind a sequence hold NaN, blocks that nobody has started the scale byte 255
        last = np.array([table[i, n - 1] for i, n in enumerate(need)])
        used = np.array([h + q - (n - 1) * page for (h, q), n in zip(lens, need)])
        at, row = np.nonzero(np.arange(page)[None, :] >= used[:, None])
        bat, blk = np.nonzero(np.arange(page // sb)[None, :] * sb >= used[:, None])
        at, row, bat, blk = (torch.from_numpy(x).cuda() for x in (last[at], row, last[bat], blk))
        for name in ("k", "v"):
            s[name + "_cache"] = _raw((pages, hkv, page, d), gen)
            s[name + "_scale"] = _scales((pages, hkv, page // sb), gen)
            s[name + "_cache"].view(torch.uint8)[at, :, row] = NEW_PAGE_BYTE
            s[name + "_scale"][bat, :, blk] = 255
        return s
    # the append: every request has the pages that its new tokens touch
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
    # one projection's output holds q, k and v of a token side by side
    qkv = torch.randn((tokens, (hq + 2 * hkv) * d), generator=gen, device="cuda")
    qkv[:, hq * d:(hq + hkv) * d] *= torch.exp(0.5 * torch.randn(hkv * d, generator=gen, device="cuda"))
    qkv = qkv.to(torch.bfloat16)
    rot, top = case["rot"], int(places.max()) + 1
    angle = torch.arange(top, dtype=torch.float64, device="cuda")[:, None] * (
        10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot))
    s = dict(case=case, pages=pages, qkv=qkv,
             q=qkv[:, :hq * d].unflatten(1, (hq, d)), k=qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
             v=qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)),
             cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(),
             positions=torch.from_numpy(places).cuda(), slot_mapping=torch.from_numpy(slots).cuda(),
             q_out=torch.zeros((tokens, hq, d), device="cuda", dtype=torch.bfloat16),
             dev_err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    for name in ("k", "v"):
        if case["op"] == "rope":
            s[name + "_cache"] = torch.randn((pages, hkv, page, d), generator=gen, device="cuda").to(torch.bfloat16)
        else:
            s[name + "_cache"] = _raw((pages, hkv, page, d), gen)
            s[name + "_scale"] = _scales((pages, hkv, page // sb), gen)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        import chunked_prefill_paged_slot_gb300 as cpsa
        if op == "rope":
            cpsa.cpp_rope_kv_cache_write(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slot_mapping"],
                                         s["k_cache"], s["v_cache"], s["q_out"], s["dev_err"],
                                         interleaved=s["case"]["inter"])
        elif op == "rope_q8":
            cpsa.cpp_rope_kv_cache_write_q8(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slot_mapping"],
                                            s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["q_out"],
                                            s["dev_err"], interleaved=s["case"]["inter"])
        else:
            if "workspace" not in s:      # a user's program keeps it from step to step
                c = s["case"]
                size = cpsa.cpp_attn_workspace_bytes(len(s["lens"]), s["q"].shape[0], c["hq"], c["hkv"], c["d"], 8)
                s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
            cpsa.cpp_chunked_prefill_attn_q8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                             s["query_lens"], s["seq_lens"], s["block_table"], s["out"],
                                             s["workspace"], s["dev_err"])
    elif op == "attn_q8":
        _plain_attention(s)
    else:
        _plain_append(s)
    if op == "attn_q8":
        return s["out"]
    got = {"q_out": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "rope_q8":
        got["k_scale"] = s["k_scale"].view(torch.float8_e8m0fnu)
        got["v_scale"] = s["v_scale"].view(torch.float8_e8m0fnu)
    return got


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


def _pow2(x):
    return (x + 127).to(torch.uint8).view(torch.float8_e8m0fnu).float()


def _need(amax):
    """The smallest x in [-117, 119] with amax <= 448 * 2^x (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(amax)
    x = e - 9 + (m > 0.875).int()
    return torch.where(amax > 0, x, torch.full_like(x, -117)).clamp(-117, 119)


def _byte(y):
    """fp32 values under their scale as e4m3 bytes."""
    y = torch.where(torch.isfinite(y), y.clamp(-448.0, 448.0), torch.full_like(y, math.nan))
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    c = s["case"]
    rot, page = c["rot"], c["page"]
    live = s["positions"] >= 0
    table = s["cos_sin"][s["positions"][live]][:, None, :]
    cos, sin = table[..., :rot // 2], table[..., rot // 2:]
    s["q_out"][live] = _rotate(s["q"][live].float(), cos, sin, rot, c["inter"]).to(torch.bfloat16)
    k, v, slot = _rotate(s["k"][live].float(), cos, sin, rot, c["inter"]), s["v"][live].float(), s["slot_mapping"][live]
    k, v, slot = k[slot >= 0], v[slot >= 0], slot[slot >= 0]
    if c["op"] == "rope":
        s["k_cache"][slot // page, :, slot % page] = k.to(torch.bfloat16)
        s["v_cache"][slot // page, :, slot % page] = v.to(torch.bfloat16)
    else:
        _plain_append_q8(k, slot, s["k_cache"], s["k_scale"], page, _sb(c))
        _plain_append_q8(v, slot, s["v_cache"], s["v_scale"], page, _sb(c))


def _plain_append_q8(x, slot, cache, scale, page, sb):
    """x [n, heads, d] to the places `slot` of cache [pages, heads, page, d] with scale [pages, heads, page / sb]."""
    cache = cache.view(torch.uint8)
    blocks = cache.view(cache.shape[0], cache.shape[1], page // sb, sb, cache.shape[3])
    at, blk = slot // page, slot % page // sb
    number = slot // sb
    amax = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(2)
    most = torch.zeros((cache.shape[0] * page // sb, x.shape[1]), device=x.device)
    most.scatter_reduce_(0, number[:, None].expand_as(amax), amax, "amax")
    fresh = torch.zeros(most.shape[0], device=x.device).scatter_reduce_(0, number, (slot % sb == 0).float(), "amax")
    fresh = (fresh[number] > 0)[:, None]
    was = scale[at, :, blk].int() - 127
    now = _need(most[number])
    now = torch.where(fresh, now, torch.maximum(now, was))
    # the other bytes of a block whose scale grows (all tokens of a block write the same)
    old = blocks[at, :, blk]
    again = _byte(old.view(torch.float8_e4m3fn).float() * _pow2(torch.where(fresh, 0, was - now).clamp(min=-127))[..., None, None])
    blocks[at, :, blk] = torch.where((~fresh & (now > was))[..., None, None], again, old)
    scale[at, :, blk] = (now + 127).to(torch.uint8)
    cache[at, :, slot % page] = _byte(x * _pow2(-now)[..., None])


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
        x = s[name + "_cache"][at].float().view(n, keys // page, hkv, page // _sb(c), _sb(c), d)
        x = x * s[name + "_scale"][at].view(torch.float8_e8m0fnu).float()[..., None, None]
        return x.view(n, keys // page, hkv, page, d).transpose(1, 2).reshape(n, hkv, keys, d)

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
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn_q8":
        return _exact_attention(s)
    rot, d = case["rot"], case["d"]
    # the rotation as a complex product
    place = s["positions"].clamp(min=0)
    turn = torch.complex(s["cos_sin"][place, :rot // 2].double(), s["cos_sin"][place, rot // 2:].double())[:, None]

    def turned(x):
        x = x.double()
        pair = x[..., :rot].unflatten(-1, (rot // 2, 2) if case["inter"] else (2, rot // 2))
        if not case["inter"]:
            pair = pair.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z if case["inter"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., rot:]], -1)

    q_out = s["q_out"].double()
    there = (s["positions"] >= 0).nonzero()[:, 0]
    q_out[there] = turned(s["q"])[there]
    got = {"q_out": q_out}
    there = ((s["positions"] >= 0) & (s["slot_mapping"] >= 0)).nonzero()[:, 0]
    slot = s["slot_mapping"][there]
    for name, x in (("k", turned(s["k"])), ("v", s["v"].double())):
        x, cache = x[there], s[name + "_cache"].double()
        if case["op"] == "rope":
            rows = cache.transpose(1, 2).reshape(-1, case["hkv"], d)
            rows[slot] = x
            got[name + "_cache"] = rows.view(-1, case["page"], case["hkv"], d).transpose(1, 2)
        else:
            got[name + "_cache"], got[name + "_scale"] = _exact_blocks(case, x, slot, cache, s[name + "_scale"])
    return got


def _exact_byte(y):
    """Nearest e4m3 value (ties to even), saturating, of 64-bit y."""
    size = y.abs().clamp(min=2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(size)) - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _exact_blocks(case, x, slot, cache, scale):
    sb, page, hkv, d = _sb(case), case["page"], case["hkv"], case["d"]
    # blocks first: [block, place, head, d]
    rows = cache.transpose(1, 2).reshape(-1, sb, hkv, d)
    power = scale.double().sub(127).transpose(1, 2).reshape(-1, hkv)
    touched, which = torch.unique(slot // sb, return_inverse=True)
    put = torch.full((len(touched), sb, hkv, d), math.nan, dtype=torch.float64, device="cuda")
    put[which, slot % sb] = x
    is_new = ~torch.isnan(put)
    high = torch.where(is_new, put.abs(), 0.0).amax((1, 3))
    want = torch.ceil(torch.log2(high / 448.0)).clamp(-117, 119)
    before = power[touched]
    restart = is_new[:, 0, 0, 0][:, None]
    after = torch.where(restart, want, torch.maximum(want, before))
    kept = rows[touched]
    moved = torch.where((~restart & (after > before))[:, None, :, None],
                        _exact_byte(kept * torch.exp2(before - after)[:, None, :, None]), kept)
    rows[touched] = torch.where(is_new, _exact_byte(put * torch.exp2(-after)[:, None, :, None]), moved)
    power[touched] = after
    return (rows.view(-1, page, hkv, d).transpose(1, 2), torch.exp2(power.view(-1, page // sb, hkv).transpose(1, 2)))


def _exact_attention(s):
    c = s["case"]
    hq, hkv, d, page, sb = c["hq"], c["hkv"], c["d"], c["page"], _sb(c)
    out, at = [], 0
    for r, (h, q) in enumerate(s["lens"]):
        n = h + q
        pages = s["block_table"][r, :-(-n // page)].long()
        got = []
        for name in ("k", "v"):
            x = s[name + "_cache"][pages].double().transpose(1, 2).reshape(-1, hkv, d)[:n]
            f = torch.exp2(s[name + "_scale"][pages].double() - 127).transpose(1, 2).reshape(-1, hkv)
            got.append((x * f.repeat_interleave(sb, 0)[:n, :, None]).transpose(0, 1).repeat_interleave(hq // hkv, 0))
        k, v = got
        z = torch.bmm(s["q"][at:at + q].double().transpose(0, 1), k.transpose(1, 2)) / math.sqrt(d)
        if q > 1:
            hidden = torch.ones((q, n), dtype=torch.bool, device="cuda").triu(h + 1)
            z.masked_fill_(hidden, -math.inf)
        out.append(torch.bmm(torch.softmax(z, -1), v).transpose(0, 1))
        at += q
    return torch.cat(out)
