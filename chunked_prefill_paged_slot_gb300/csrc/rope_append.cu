// rope_append.cu -- the rotary KV append: rotate the new tokens' q and k by
// their positions, write the rotated q, and append k and v to the paged cache,
// in one pass over the projection's output. Three cache formats: bf16; e4m3
// bytes with a power-of-two scale per (page, kv head, block of SB tokens),
// SB = min(16, page_size); and 4-bit codes with a scale per place, kv head and 16
// columns (q4.cuh). With NORM every q and k head is first brought to unit mean square
// and multiplied by its weights.
//
// Rotation of a pair (a, b) by the angle t of its position:
//   (a cos t - b sin t, b cos t + a sin t),
// each product and each sum rounded to fp32 on its own (no fused multiply-add):
// one fixed result whatever the compiler contracts, so that a quantised byte next
// to a rounding border does not depend on the build. cos t and sin t come from the
// caller's fp32 table.
//
// A unit is 16 columns of one head of one token, the two 16-byte vectors that one
// thread reads, rotates and writes: columns [8u, 8u + 8) and their partners
// [rot/2 + 8u, ...) (half-split pairs), or columns [16u, 16u + 16) (interleaved
// pairs, and the columns from rot on, which pass through). Reading and writing the
// same bytes in one thread is what lets q_out be q itself.
//
// Bound by memory: 2 bytes in and 2 (or 1) out per element, and the table's row. The
// bf16 append of a 32768-token prompt (32/8 heads, D 128, 823 MB) takes 123 us, 6.7 TB/s
// or 99 % of a plain copy's rate; small calls are bound by latency (one token: 2 us
// replayed among others, 11 us a call).
#include "common.cuh"
#include "kernels.cuh"
#include "q4.cuh"
#include "q8.cuh"

namespace cpsa {

namespace {

constexpr int kRopeThreads = 128;

// The two vectors of unit u: their first columns.
__device__ __forceinline__ void unit_cols(int u, int rot, bool inter, int &c0, int &c1)
{
    const bool split = !inter && u < (rot >> 4);
    c0 = split ? 8 * u : 16 * u;
    c1 = split ? (rot >> 1) + 8 * u : 16 * u + 8;
}

__device__ __forceinline__ void widen8(const uint4 &x, float (&f)[8])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 narrow8(const float (&f)[8])
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void load8(const float *p, float (&f)[8])
{
    const float4 x = __ldg(reinterpret_cast<const float4 *>(p)), y = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
}

// A byte loaded where this stands (it may have been written by an earlier round of this
// warp, so not through the read-only path).
__device__ __forceinline__ uint32_t load_byte_here(const uint8_t *p)
{
    uint32_t v;
    asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void rotate_pair(float &a, float &b, float c, float s)
{
    const float ra = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    const float rb = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = ra;
    b = rb;
}

// x0, x1: the unit's 16 columns in order of its two vectors.
__device__ __forceinline__ void rotate_unit(float (&x0)[8], float (&x1)[8], const float (&c)[8], const float (&s)[8],
                                            bool inter)
{
    if (inter) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rotate_pair(x0[2 * i], x0[2 * i + 1], c[i], s[i]);
            rotate_pair(x1[2 * i], x1[2 * i + 1], c[4 + i], s[4 + i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) rotate_pair(x0[i], x1[i], c[i], s[i]);
    }
}

// What a token's position says: 0 rotate and write, 1 padding (skipped whole), 2 out of range.
__device__ __forceinline__ int position_state(const RopeParams &p, int64_t t, int64_t &pos)
{
    pos = 0;
    if (p.rot == 0)
        return 0;
    pos = __ldg(p.positions + t);
    return pos < 0 ? 1 : (pos >= p.max_positions ? 2 : 0);
}

// Head norm: y_c = x_c / sqrt(mean_c x_c^2 + eps) * w_c, in fp32. The D/16 threads of a head
// are neighbours in a warp: each sums its 16 squares (exact products of bf16 numbers), a
// butterfly adds up the threads', in an order that does not depend on anything. (By rsqrtf,
// within two last places: a 32768-token prompt, 32/8 heads, D 128, takes 146 us into the bf16
// cache, 150 us by a root and a division, 123 us without norms; 179 and 148 us into the 8-bit, 168 and
// 139 into the 4-bit cache. 2048 tokens into bf16 from HBM 14.2 us, 11.5 without norms, 7.7 by their bytes:
// the position, the slot, the rows, the sum and the weights wait for one another.)
__device__ __forceinline__ float squares8(const uint4 &x)
{
    float f[8], a = 0.f;
    widen8(x, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaf(f[i], f[i], a);
    return a;
}

template <int D>
__device__ __forceinline__ float inverse_rms(const uint4 &v0, const uint4 &v1, float eps, uint32_t mask)
{
    float a = squares8(v0) + squares8(v1);
#pragma unroll
    for (int o = D / 32; o > 0; o >>= 1) a += __shfl_xor_sync(mask, a, o);
    return rsqrtf(fmaf(a, 1.f / D, eps));
}

__device__ __forceinline__ void scale8(float (&x)[8], float f, const float (&w)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * f * w[i];
}

__device__ __forceinline__ void scale8(float (&x)[8], float f, const float *w)
{
    float k[8];
    load8(w, k);
    scale8(x, f, k);
}

// What rope_heads does with k and v.
enum { kNoKv, kKvBf16, kKvQ4 };

// A unit of a k head whose 16 columns are two vectors of eight from c0 and c1 on, of two
// groups: the amax bits of each vector's other half of its group. Vectors of eight are
// numbered along the head; number i sits at (unit, which) = (i, 0) and (i - R, 1) for the R
// split units' first and second vectors, (i / 2, i & 1) behind them.
template <int D>
__device__ __forceinline__ void group_partners(uint32_t m0, uint32_t m1, int u, int rot, bool inter, uint32_t mask,
                                               uint32_t &o0, uint32_t &o1)
{
    if (inter || rot == 0) {
        o0 = m1;
        o1 = m0;
        return;
    }
    if ((rot & 31) == 0) {   // both halves of a group sit in the same place of two neighbours
        const uint32_t a = __shfl_xor_sync(mask, m0, 1), b = __shfl_xor_sync(mask, m1, 1);
        const bool split = u < (rot >> 4);
        o0 = split ? a : m1;
        o1 = split ? b : m0;
        return;
    }
    const int R = rot >> 4;
    int c0, c1;
    unit_cols(u, rot, inter, c0, c1);
    auto fetch = [&](int i) -> uint32_t {
        const int from = i < R ? i : (i < 2 * R ? i - R : i >> 1);
        const bool second = i < R ? false : (i < 2 * R ? true : (i & 1) != 0);
        const uint32_t a = __shfl_sync(mask, m0, from, D / 16), b = __shfl_sync(mask, m1, from, D / 16);
        return second ? b : a;
    };
    o0 = fetch((c0 >> 3) ^ 1);
    o1 = fetch((c1 >> 3) ^ 1);
}

// One unit column u of HPT consecutive heads of one token: q heads, then (KV: into the
// bf16 or the 4-bit cache) k heads, then v heads. The table's values are loaded once for
// all of them, and every head's vectors are in flight before the first is used.
template <int D, int HPT, int KV, bool NORM>
__device__ __forceinline__ void rope_heads(const RopeParams &p, int64_t t, int head0, int u)
{
    constexpr bool WITH_KV = KV != kNoKv;
    const int heads = WITH_KV ? p.Hq + 2 * p.Hkv : p.Hq;
    // the head's threads, which have the same way through here
    const uint32_t mask = (D == 128 ? 0xffu : 0xfu) << (threadIdx.x & 31 & ~(D / 16 - 1));
    int64_t pos;
    const int state = position_state(p, t, pos);
    if (state != 0) {
        if (state == 2 && head0 == 0 && u == 0)
            set_dev_error(p.dev_err, CPSA_DEV_POSITION_OUT_OF_RANGE);
        return;
    }
    int64_t slot = -1;
    if (WITH_KV && head0 + HPT > p.Hq) {
        slot = __ldg(p.slot_mapping + t);
        if (slot >= p.num_pages * (int64_t)p.page_size) {
            if (head0 + HPT >= heads && u == 0)
                set_dev_error(p.dev_err, CPSA_DEV_SLOT_OUT_OF_RANGE);
            slot = -1;
        }
    }
    int c0, c1;
    unit_cols(u, p.rot, p.inter, c0, c1);
    const bool turn = u < (p.rot >> 4);
    uint4 v0[HPT], v1[HPT];
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
        const int h = head0 + i;
        if (h >= heads || (h >= p.Hq && slot < 0))
            continue;
        const __nv_bfloat16 *src = h < p.Hq ? p.q + t * p.q_stride + h * D
                                   : h < p.Hq + p.Hkv ? p.k + t * p.k_stride + (h - p.Hq) * D
                                                      : p.v + t * p.v_stride + (h - p.Hq - p.Hkv) * D;
        const bool whole = KV == kKvQ4 && h >= p.Hq + p.Hkv;   // a v unit of the 4-bit cache is one group
        v0[i] = *reinterpret_cast<const uint4 *>(src + (whole ? 16 * u : c0));
        v1[i] = *reinterpret_cast<const uint4 *>(src + (whole ? 16 * u + 8 : c1));
    }
    float c[8], s[8];
    if (turn) {
        load8(p.cos_sin + pos * p.rot + 8 * u, c);
        load8(p.cos_sin + pos * p.rot + (p.rot >> 1) + 8 * u, s);
    }
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
        const int h = head0 + i;
        if (h >= heads || (h >= p.Hq && slot < 0))
            continue;
        const bool normed = NORM && h < p.Hq + p.Hkv;
        const bool four = KV == kKvQ4 && h >= p.Hq;
        if ((turn && h < p.Hq + p.Hkv) || normed || four) {
            float x0[8], x1[8];
            widen8(v0[i], x0);
            widen8(v1[i], x1);
            if (normed) {
                const float f = inverse_rms<D>(v0[i], v1[i], p.eps, mask);
                const float *w = h < p.Hq ? p.q_weight : p.k_weight;
                scale8(x0, f, w + c0);
                scale8(x1, f, w + c1);
            }
            if (turn && h < p.Hq + p.Hkv)
                rotate_unit(x0, x1, c, s, p.inter);
            if (four) {
                const bool is_k = h < p.Hq + p.Hkv;
                const int kvh = is_k ? h - p.Hq : h - p.Hq - p.Hkv;
                const int64_t row = ((slot >> p.lg_page) * p.Hkv + kvh) * p.page_size + (slot & (p.page_size - 1));
                uint8_t *codes = reinterpret_cast<uint8_t *>(is_k ? p.k_cache : p.v_cache) + row * (D / 2);
                uint8_t *scales = (is_k ? p.k_scale : p.v_scale) + row * (D / kQ4Group);
                const uint32_t m0 = q4_amax(x0), m1 = q4_amax(x1);
                if (!is_k) {
                    const Q4Scale f(max(m0, m1));
                    *reinterpret_cast<uint2 *>(codes + 8 * u) = make_uint2(q4_codes(x0, f), q4_codes(x1, f));
                    scales[u] = f.byte;
                } else {
                    uint32_t o0, o1;
                    group_partners<D>(m0, m1, u, p.rot, p.inter, mask, o0, o1);
                    const Q4Scale f0(max(m0, o0)), f1(max(m1, o1));
                    *reinterpret_cast<uint32_t *>(codes + (c0 >> 1)) = q4_codes(x0, f0);
                    *reinterpret_cast<uint32_t *>(codes + (c1 >> 1)) = q4_codes(x1, f1);
                    if ((c0 & 8) == 0)
                        scales[c0 >> 4] = f0.byte;
                    if ((c1 & 8) == 0)
                        scales[c1 >> 4] = f1.byte;
                }
                continue;
            }
            v0[i] = narrow8(x0);
            v1[i] = narrow8(x1);
        }
        __nv_bfloat16 *dst;
        if (h < p.Hq) {
            dst = p.q_out + (t * p.Hq + h) * D;
        } else {
            const bool is_k = h < p.Hq + p.Hkv;
            const int kvh = is_k ? h - p.Hq : h - p.Hq - p.Hkv;
            const int64_t page = slot >> p.lg_page;
            dst = reinterpret_cast<__nv_bfloat16 *>(is_k ? p.k_cache : p.v_cache) +
                  ((page * p.Hkv + kvh) * p.page_size + (slot & (p.page_size - 1))) * D;
        }
        *reinterpret_cast<uint4 *>(dst + c0) = v0[i];
        *reinterpret_cast<uint4 *>(dst + c1) = v1[i];
    }
}

// Items (token, group of HPT heads), D/16 threads each, units fastest: the eight
// threads of a 128-column head read 128 consecutive bytes twice.
template <int D, int HPT, int KV, bool NORM>
__device__ __forceinline__ void rope_items(const RopeParams &p, int64_t first, int64_t step)
{
    constexpr int UPH = D / 16;
    const int groups = ((KV != kNoKv ? p.Hq + 2 * p.Hkv : p.Hq) + HPT - 1) / HPT;
    const int64_t total = p.num_tokens * groups;
    for (int64_t i = first / UPH; i < total; i += step / UPH)
        rope_heads<D, HPT, KV, NORM>(p, i / groups, (int)(i % groups) * HPT, (int)(first % UPH));
}

// Seven blocks an SM (72 registers) with norms or 4 bits: a 32768-token prompt (32/8 heads, D 128) into
// the 4-bit cache takes 139 us, 158 us with the 84 registers the compiler takes by itself. (With norms and
// 4 bits, two heads a thread, that spills 86 bytes.)
template <int D, int HPT, int KV, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, KV == kKvQ4 || NORM ? 7 : 0) rope_append_kernel(const RopeParams p)
{
    pdl_trigger();
    pdl_wait();
    rope_items<D, HPT, KV, NORM>(p, (int64_t)blockIdx.x * kRopeThreads + threadIdx.x,
                                 (int64_t)gridDim.x * kRopeThreads);
}

// ---------------------------------------------------------------------------
// The 8-bit cache. value = byte * 2^x, x the block's scale exponent (its scale
// byte - 127). Tokens that one call puts into one block, neighbours in the call
// with ascending slots, form a run; need = the smallest x with amax <= 448 * 2^x
// over the run's finite values, within [kQ8MinExp, kQ8MaxExp]. A run that holds
// the block's first place starts the block over (x = need); any other keeps
// x = max(need, old x), and where that grows, the block's other bytes are rounded
// to the new scale -- a shift of their exponent, which loses only what falls
// under the coarser subnormal step. Powers of two make every stored value exact
// in bf16, and exponents between -117 and 119 keep every such value a normal
// fp32 number, subnormal bytes included.
//
// One warp does the runs that start in one window of 16 tokens, for one kv head
// and one of k and v: every run has one owner, so neither the scale nor the
// rewriting of a block is raced for and the result does not depend on timing.
// It takes up to 16 rows at a time (D/16 lanes a row), whole runs only, all their
// loads in flight together; a row's slot and run live in the lane of its number.
// ---------------------------------------------------------------------------
constexpr int kQ8Rows = 16;

// Smallest x with a <= 448 * 2^x (448 = 1.75 * 2^8), clamped.
__device__ __forceinline__ int need_exponent(float a)
{
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(kQ8MinExp, min(kQ8MaxExp, e));
}

// 2^x, -127 <= x <= 127 (the smallest of them a subnormal number)
__device__ __forceinline__ float exp2_int(int x)
{
    return __uint_as_float(x > -127 ? (uint32_t)(x + 127) << 23 : 0x400000u);
}

// Two values under their scale as e4m3 bytes: nearest even, saturating (infinities
// too), NaN as NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// An infinity as NaN; anything else as it is.
__device__ __forceinline__ float inf_to_nan(float x) { return fmaf(x, 0.f, x); }

__device__ __forceinline__ uint32_t rescale_bytes(uint32_t w, uint32_t f16x2_factor)
{
    // e4m3 -> f16 is exact, and so is the product wherever it can still round to a
    // nonzero byte (a byte's last place times 2^-15 is f16's smallest number)
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint16_t b = (uint16_t)(w >> (16 * i));
        uint32_t h;
        uint16_t r;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(b));
        asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h) : "r"(f16x2_factor));
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
        out |= (uint32_t)r << (16 * i);
    }
    return out;
}

template <int D, bool NORM>
__device__ __forceinline__ void append_q8_window(const RopeParams &p, int64_t window, int job, int lane)
{
    constexpr int LPR = D / 16;              // lanes per row
    constexpr int RPP = 32 / LPR;            // rows per pass
    constexpr int PASSES = kQ8Rows / RPP;
    const bool is_k = job < p.Hkv;
    const int kvh = is_k ? job : job - p.Hkv;
    const int rsub = lane / LPR, u = lane % LPR;
    const int64_t slots = p.num_pages << p.lg_page;
    const int lg_sb = min(4, p.lg_page);
    const int64_t w0 = window * kQ8Rows;

    // The window's rows are asked for before anything is known of their slots: nearly
    // always they are the rows to do (else they are loaded again), and the two latencies
    // overlap.
    uint4 v0[PASSES], v1[PASSES];
    float norm[PASSES];                      // NORM: 1 / root mean square of the k rows
    int c0, c1;
    unit_cols(u, is_k ? p.rot : 0, p.inter, c0, c1);
    const __nv_bfloat16 *src = is_k ? p.k + kvh * D : p.v + kvh * D;
    const int64_t stride = is_k ? p.k_stride : p.v_stride;
    auto load_rows = [&](int64_t first) {
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
            const int64_t t = first + q * RPP + rsub;
            v0[q] = v1[q] = make_uint4(0, 0, 0, 0);
            if (t < p.num_tokens) {
                v0[q] = __ldcs(reinterpret_cast<const uint4 *>(src + t * stride + c0));
                v1[q] = __ldcs(reinterpret_cast<const uint4 *>(src + t * stride + c1));
            }
        }
    };
    load_rows(w0);

    // slot and position of token t, or -1 where nothing is to be written
    auto slot_of = [&](int64_t t, bool report, int64_t &pos) -> int64_t {
        pos = 0;
        if (t < 0 || t >= p.num_tokens)
            return -1;
        const int state = position_state(p, t, pos);
        const int64_t s = __ldg(p.slot_mapping + t);
        if (state != 0) {
            if (state == 2 && report)
                set_dev_error(p.dev_err, CPSA_DEV_POSITION_OUT_OF_RANGE);
            return -1;
        }
        if (s >= slots) {
            if (report)
                set_dev_error(p.dev_err, CPSA_DEV_SLOT_OUT_OF_RANGE);
            return -1;
        }
        return s;
    };
    // lane l looks at token w0 + l: the window and the up to 15 tokens behind it
    // that can still belong to its last run
    int64_t pos, pos_before;
    const int64_t slot = slot_of(w0 + lane, job == 0 && lane < kQ8Rows, pos);
    int64_t before = __shfl_up_sync(0xffffffffu, slot, 1);
    if (lane == 0)
        before = slot_of(w0 - 1, false, pos_before);
    const bool live = slot >= 0;
    const bool joins = live && before >= 0 && (before >> lg_sb) == (slot >> lg_sb) && before < slot;
    const uint32_t lead = __ballot_sync(0xffffffffu, live && !joins);
    const uint32_t cont = __ballot_sync(0xffffffffu, joins);
    // the rows to do: runs whose first token is in the window
    uint32_t todo = lead & 0xffffu;
    int loaded = 0;   // v0, v1 hold the rows from this one on
    while (todo) {
        // the next whole runs, at most kQ8Rows rows from the first one's start (a run is
        // at most SB <= 16 rows long, so there is always at least one)
        const int base = __ffs(todo) - 1;
        uint32_t leads = 0;
        int rows = 0;
        while (todo) {
            const int b = __ffs(todo) - 1;
            const uint32_t after = b < 31 ? ~(cont >> (b + 1)) : ~0u;
            const int len = __ffs(after);      // the leader and the joining rows right behind it
            if (b + len - base > kQ8Rows)
                break;
            leads |= 1u << (b - base);
            rows = b + len - base;
            todo &= todo - 1;
        }
        // row i's slot in lane i; rows between runs (padding) have -1
        const int64_t rslot = __shfl_sync(0xffffffffu, slot, (base + lane) & 31);
        const bool mine = lane < rows && rslot >= 0;
        if (base != loaded)
            load_rows(w0 + base);
        loaded = base;
        const int64_t rpos = __shfl_sync(0xffffffffu, pos, (base + lane) & 31);
        // the rows' places, and the scales of blocks that are not started over: asked for here,
        // ahead of the rotation, they are there when the new scale needs them (128 single
        // tokens in a graph 10.3 -> 8.3 us, 2048 rows 16.6 -> 12.3 us)
        const uint32_t upto = leads & (0xffffffffu >> (31 - lane));
        const int start = upto ? 31 - __clz(upto) : 0;
        const uint32_t minemask = __ballot_sync(0xffffffffu, mine);
        const int64_t page = rslot >> p.lg_page;
        const int off = (int)rslot & (p.page_size - 1);
        uint8_t *scale = (is_k ? p.k_scale : p.v_scale) +
                         (page * p.Hkv + kvh) * (p.page_size >> lg_sb) + (off >> lg_sb);
        uint8_t *bytes = reinterpret_cast<uint8_t *>(is_k ? p.k_cache : p.v_cache) +
                         (page * p.Hkv + kvh) * (int64_t)p.page_size * D;
        bool kept = false;
        uint32_t was_byte = 0;
        if (mine) {
            kept = ((int)__shfl_sync(minemask, off, start) & ((1 << lg_sb) - 1)) != 0;
            if (kept)
                was_byte = load_byte_here(scale);
        }
        // this lane's 16 values of pass q, rotated; on: its row is one to do (any other's
        // position may be no row of the table)
        auto values = [&](int q, bool on, float (&x0)[8], float (&x1)[8]) {
            widen8(v0[q], x0);
            widen8(v1[q], x1);
            if (NORM && is_k) {
                scale8(x0, norm[q], p.k_weight + c0);
                scale8(x1, norm[q], p.k_weight + c1);
            }
            const int64_t at = __shfl_sync(0xffffffffu, rpos, q * RPP + rsub);
            if (on && is_k && u < (p.rot >> 4)) {
                float c[8], s[8];
                load8(p.cos_sin + at * p.rot + 8 * u, c);
                load8(p.cos_sin + at * p.rot + (p.rot >> 1) + 8 * u, s);
                rotate_unit(x0, x1, c, s, p.inter);
            }
        };
        if (NORM && is_k) {
#pragma unroll
            for (int q = 0; q < PASSES; ++q) norm[q] = inverse_rms<D>(v0[q], v1[q], p.eps, 0xffffffffu);
        }
        // 1. the rows' largest finite magnitudes. Infinities, which neither count nor saturate
        // but become NaN, are rare: whether there are any is seen from the maxima, and only
        // then is every value looked at for itself. (A maximum passes over NaN.)
        float rowmax = 0.f;
        bool inf = false;
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
            const int row = q * RPP + rsub;
            const bool on = __shfl_sync(0xffffffffu, (int)mine, row) != 0;
            float m = 0.f;
            if (is_k) {
                float x0[8], x1[8];
                values(q, on, x0, x1);
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(x0[i]), fabsf(x1[i])));
                if (m == INFINITY) {
                    m = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float a = fabsf(x0[i]), b = fabsf(x1[i]);
                        m = fmaxf(m, a < INFINITY ? a : 0.f);      // false for NaN
                        m = fmaxf(m, b < INFINITY ? b : 0.f);
                    }
                    inf = true;
                }
            } else {
                m = fmaxf(bf16x8_amax(v0[q], inf), bf16x8_amax(v1[q], inf));
            }
            m = on ? m : 0.f;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            // to the lane of the row's number
            const float got = __shfl_sync(0xffffffffu, m, (lane % RPP) * LPR);
            if (lane / RPP == q)
                rowmax = got;
        }
        inf = __any_sync(0xffffffffu, inf);
        // 2. each run's maximum (rows of a run are neighbours), its old and its new scale
        float runmax = mine ? rowmax : 0.f;
#pragma unroll
        for (int o = 1; o < kQ8Rows; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, runmax, o);
            if (lane - o >= start)
                runmax = fmaxf(runmax, y);
        }
        // the run's last row holds its maximum: the row before the next leader or gap
        const uint32_t stops = (leads | ~minemask) & (lane < 31 ? 0xfffffffeu << lane : 0u);
        const int last = stops ? __ffs(stops) - 2 : 31;
        runmax = __shfl_sync(0xffffffffu, runmax, last);
        int x = 0, grow = 0;
        if (mine) {
            x = need_exponent(runmax);
            if (kept) {
                // (another writer's may be above kQ8MaxExp; 255, which stands for none, as 254)
                const int was = min((int)was_byte - 127, 127);
                grow = max(0, x - was);
                x = max(x, was);
            }
        }
        __syncwarp();
        if (mine && lane == start)
            *scale = (uint8_t)(x + 127);
        // 3. blocks whose scale grew: round their other bytes to it
        uint32_t grown = __ballot_sync(0xffffffffu, mine && lane == start && grow > 0);
        while (grown) {
            const int r = __ffs(grown) - 1;
            grown &= grown - 1;
            const uint32_t put = __reduce_or_sync(0xffffffffu, mine && start == r ? 1u << (off & ((1 << lg_sb) - 1)) : 0u);
            const int g = min(__shfl_sync(0xffffffffu, grow, r), 24);
            const int first = __shfl_sync(0xffffffffu, off, r) & ~((1 << lg_sb) - 1);
            uint8_t *blk = reinterpret_cast<uint8_t *>(
                               __shfl_sync(0xffffffffu, (unsigned long long)reinterpret_cast<uintptr_t>(bytes), r)) +
                           (int64_t)first * D;
            // 2^-g as an f16 pair (a subnormal f16 below 2^-14)
            const uint32_t f = g <= 14 ? (uint32_t)(15 - g) << 10 : 1u << (24 - g);
            const uint32_t f2 = f | f << 16;
            for (int v = lane; v < (D / 16) << lg_sb; v += 32) {
                if ((put >> (v / (D / 16))) & 1u)
                    continue;
                uint4 b = *reinterpret_cast<uint4 *>(blk + v * 16);
                b.x = rescale_bytes(b.x, f2);
                b.y = rescale_bytes(b.y, f2);
                b.z = rescale_bytes(b.z, f2);
                b.w = rescale_bytes(b.w, f2);
                *reinterpret_cast<uint4 *>(blk + v * 16) = b;
            }
        }
        // 4. the new rows' bytes
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
            const int row = q * RPP + rsub;
            const bool on = __shfl_sync(0xffffffffu, (int)mine, row) != 0;
            const float f = exp2_int(-__shfl_sync(0xffffffffu, x, row));
            uint8_t *dst = reinterpret_cast<uint8_t *>(__shfl_sync(
                0xffffffffu, (unsigned long long)reinterpret_cast<uintptr_t>(bytes + (int64_t)off * D), row));
            float x0[8], x1[8];
            values(q, on, x0, x1);
            if (!on)
                continue;
            if (inf) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x0[i] = inf_to_nan(x0[i]);
                    x1[i] = inf_to_nan(x1[i]);
                }
            }
            uint32_t b0[2], b1[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                b0[i] = e4m3x2(x0[4 * i] * f, x0[4 * i + 1] * f) | e4m3x2(x0[4 * i + 2] * f, x0[4 * i + 3] * f) << 16;
                b1[i] = e4m3x2(x1[4 * i] * f, x1[4 * i + 1] * f) | e4m3x2(x1[4 * i + 2] * f, x1[4 * i + 3] * f) << 16;
            }
            *reinterpret_cast<uint2 *>(dst + c0) = make_uint2(b0[0], b0[1]);
            *reinterpret_cast<uint2 *>(dst + c1) = make_uint2(b1[0], b1[1]);
        }
        __syncwarp();
    }
}

// Blocks [0, kv_blocks): one warp per (window, kv head, k or v), heads fastest (the
// table's rows of a window are shared through L1); the rest: the q heads.
// Five blocks an SM (96 registers): a 32768-token prompt (32/8 heads, D 128, 756 MB, 111 us
// at a plain copy's rate) takes 148 us; 161 us with the 116 registers the compiler takes by
// itself, 159, 147, 151 and 194 us with four, six, seven and eight blocks. (181 us when the
// rows were asked for only once their slots were known and kept rotated in registers.)
template <int D, int HPT, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, 5) rope_append_q8_kernel(const RopeParams p, int kv_blocks)
{
    pdl_trigger();
    pdl_wait();
    if ((int)blockIdx.x < kv_blocks) {
        const int64_t windows = (p.num_tokens + kQ8Rows - 1) / kQ8Rows;
        const int64_t w = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
        if (w < windows * 2 * p.Hkv)
            append_q8_window<D, NORM>(p, w / (2 * p.Hkv), (int)(w % (2 * p.Hkv)), threadIdx.x & 31);
    } else {
        rope_items<D, HPT, kNoKv, NORM>(p, (int64_t)(blockIdx.x - kv_blocks) * kRopeThreads + threadIdx.x,
                                        (int64_t)(gridDim.x - kv_blocks) * kRopeThreads);
    }
}

// Heads per thread: one while a single wave of threads holds every unit (the
// fewest dependent steps, which is all that counts there), else two (four beside the
// 8-bit cache's windows, whose registers leave fewer warps to keep loads in flight): the
// table's values are loaded once for them. A 32768-token prompt into the bf16 cache takes
// 123 us with two and 127 with four, into the 8-bit cache 161 and 148.
constexpr int kRopeHeads = 2, kRopeHeadsQ8 = 4;

template <int D, bool NORM>
cudaError_t launch_rope_t(const RopeParams &p, int bits, int num_sms, cudaStream_t s)
{
    const bool q8 = bits == 8;
    const int heads = q8 ? p.Hq : p.Hq + 2 * p.Hkv;
    const int many = q8 ? kRopeHeadsQ8 : kRopeHeads;
    const bool one = p.num_tokens * heads * (D / 16) <= (int64_t)num_sms * 1024;
    const int64_t items = p.num_tokens * (one ? heads : (heads + many - 1) / many) * (D / 16);
    int64_t blocks = (items + kRopeThreads - 1) / kRopeThreads;
    if (blocks > (int64_t)num_sms * 64)
        blocks = (int64_t)num_sms * 64;
    if (!q8) {
        auto k = bits == 4 ? (one ? rope_append_kernel<D, 1, kKvQ4, NORM> : rope_append_kernel<D, kRopeHeads, kKvQ4, NORM>)
                           : (one ? rope_append_kernel<D, 1, kKvBf16, NORM> : rope_append_kernel<D, kRopeHeads, kKvBf16, NORM>);
        return launch_pdl(false, k, dim3((unsigned)blocks), dim3(kRopeThreads), 0, s, p);
    }
    const int64_t warps = (p.num_tokens + kQ8Rows - 1) / kQ8Rows * 2 * p.Hkv;
    const int64_t kv_blocks = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    if (kv_blocks + blocks > 0x7fffffff)
        return cudaErrorInvalidValue;
    return launch_pdl(false, one ? rope_append_q8_kernel<D, 1, NORM> : rope_append_q8_kernel<D, kRopeHeadsQ8, NORM>,
                      dim3((unsigned)(kv_blocks + blocks)), dim3(kRopeThreads), 0, s, p, (int)kv_blocks);
}

// Rows of the 4-bit cache as bf16, gathered by slot: a thread takes one group of 16 columns of
// one token's k and v of one head, and stores its 32 bytes at once (WIDE: k and v on 32-byte
// boundaries) or in two halves. Bound by memory: 0.56 bytes in and 2 out per element. (25.6 k
// rows of 8 heads, D 128, 135 MB: over several such inputs in turn 24.9 us, 27.1 us with eight
// columns a thread; 131 k rows 73 and 83 us. Where one call's rows stay in L2 eight columns are the
// faster, 19.4 instead of 22.4 us; rows of a cache are rarely there. 30.6 us in two halves.)
constexpr int kReadThreads = 256;

template <bool WIDE>
__device__ __forceinline__ void store_group(__nv_bfloat16 *dst, const uint4 &a, const uint4 &b)
{
    if (WIDE) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                     "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = a;
        reinterpret_cast<uint4 *>(dst)[1] = b;
    }
}

template <int D, bool WIDE>
__global__ void __launch_bounds__(kReadThreads) read_q4_kernel(const ReadQ4Params p)
{
    constexpr int TPR = D / kQ4Group;   // threads per row
    pdl_trigger();
    pdl_wait();
    const int64_t t = (int64_t)blockIdx.x * (kReadThreads / TPR) + threadIdx.x / TPR;
    const int u = threadIdx.x % TPR, h = blockIdx.y;
    if (t >= p.num_tokens)
        return;
    const int64_t slot = __ldg(p.slot_mapping + t);
    if (slot < 0)
        return;
    if (slot >= p.num_pages << p.lg_page) {
        if (h == 0 && u == 0)
            set_dev_error(p.dev_err, CPSA_DEV_SLOT_OUT_OF_RANGE);
        return;
    }
    const int64_t row = (((slot >> p.lg_page) * p.Hkv + h) << p.lg_page) + (slot & ((1 << p.lg_page) - 1));
    const uint2 kc = __ldg(reinterpret_cast<const uint2 *>(p.k_cache + row * (D / 2)) + u);
    const uint2 vc = __ldg(reinterpret_cast<const uint2 *>(p.v_cache + row * (D / 2)) + u);
    const uint32_t ks = __ldg(p.k_scale + row * TPR + u), vs = __ldg(p.v_scale + row * TPR + u);
    const int64_t at = (t * p.Hkv + h) * D + kQ4Group * u;
    store_group<WIDE>(p.k + at, q4_bf16x8(kc.x, ks), q4_bf16x8(kc.y, ks));
    store_group<WIDE>(p.v + at, q4_bf16x8(vc.x, vs), q4_bf16x8(vc.y, vs));
}

template <int D>
cudaError_t launch_read_t(const ReadQ4Params &p, cudaStream_t s)
{
    constexpr int rows = kReadThreads / (D / kQ4Group);
    const bool wide = ((reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v)) & 31u) == 0;
    return launch_pdl(false, wide ? read_q4_kernel<D, true> : read_q4_kernel<D, false>, dim3((unsigned)((p.num_tokens + rows - 1) / rows), (unsigned)p.Hkv),
                      dim3(kReadThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams &p, int head_dim, int bits, int num_sms, cudaStream_t s)
{
    if (p.num_tokens == 0)
        return cudaSuccess;
    const bool norm = p.k_weight != nullptr;
    if (head_dim == 128)
        return norm ? launch_rope_t<128, true>(p, bits, num_sms, s) : launch_rope_t<128, false>(p, bits, num_sms, s);
    return norm ? launch_rope_t<64, true>(p, bits, num_sms, s) : launch_rope_t<64, false>(p, bits, num_sms, s);
}

cudaError_t launch_read_q4(const ReadQ4Params &p, int head_dim, cudaStream_t s)
{
    if (p.num_tokens == 0)
        return cudaSuccess;
    return head_dim == 128 ? launch_read_t<128>(p, s) : launch_read_t<64>(p, s);
}

}  // namespace cpsa
