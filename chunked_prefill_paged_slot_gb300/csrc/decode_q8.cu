// decode_q8.cu -- split-KV attention of decode rows (query_len == 1) over the
// 8-bit paged cache (e4m3 bytes, a power-of-two scale per block of SB places and kv
// head). Bound by HBM: every byte of the row's context is read once, for all the q
// heads of its kv head at once.
//
// softmax(scale * q K^T) V over keys [key0, key1) of one row, for HG kv heads (8, 4,
// 2 or 1 by what divides the head count: the more heads of a page an item takes, the
// longer the contiguous reads) and their G q heads each.
//
// CTA (288 threads, persistent over the plan's items):
//   warp 8     producer: stages of KS = 256 / HG keys of HG heads, K and V, one TMA
//              box per page (or 64 rows of one) and tensor covering the heads; page
//              numbers a window of stages ahead, scale bytes two stages ahead,
//              handed over in shared memory with the stage.
//   warps 0..7 warp w: kv head w % HG of the group, keys [32 (w / HG), + 32) of every
//              stage. The 8 / HG warps of a head meet in shared memory at the end.
//
// Arithmetic. e4m3 -> f16 is exact, so the bytes go into mma.sync m16n8k16 (f16 in,
// fp32 sums) unscaled, one cvt per two bytes, and the scales into the few numbers per
// key: the fp32 scores are multiplied by the key block's, the fp32 probabilities by
// the value block's before they are rounded to f16. Of q, each row is brought to f16
// by a power of two that puts its largest element in [2^14, 2^15); what that drops
// is under 2^-39 of the row's largest. The probabilities p * 2^(x_block - X + 15), X
// the largest value exponent so far (O is rescaled when it rises), keep f16's 11 bits
// down to 2^-29 of the largest: more than bf16's 8 wherever they count.
//
// Keys are the M rows of the scores (16 keys x 16 columns times 16 columns x 8 heads) and
// columns those of the output (16 columns x 16 keys times 16 keys x 8 heads), heads the N
// columns of both: eight of them fill an n tile, where as M rows they would leave half of
// every MMA empty (that way round the kernel was bound by mma.sync: 2330 of 2850 clocks a
// stage). The probabilities pass from one to the other by 8 x 8 transposes in registers.
//
// Measured (32/8 heads, D 128, pages of 16): 128 rows of 2600 to 5200 keys, 1.05 GB, in
// 170 us, 6.2 TB/s or 91 % of a plain copy's rate; the rest of a call's 195 us is the plan,
// the empty chunk launch and the combine. Stages of 64 KB, three of them (two where the
// merge needs room), keep 128 to 192 KB a SM in flight.
//
// Shared memory layouts and fragments. A row of a stage is D bytes, its 16-byte
// chunks swizzled by TMA. The k index of an mma is a free relabelling of columns
// (scores) or keys (P V), the m index of keys or columns, so the fragments are chosen
// for the loads: lane (g, t) = (lane / 4, lane % 4) takes, of key kappa(g) of each
// eight, the chunks t (and t + 4): 16-byte loads that hold four whole k steps; of V the
// keys kappa(2t), kappa(2t + 1) of each eight, D/8 consecutive columns at chi(g), the
// two keys' bytes interleaved by byte permutes into (key, key) pairs. kappa and chi
// are such that every such load of a warp is free of bank conflicts.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.cuh"
#include "plan.cuh"
#include "q8.cuh"

namespace cpsa {

namespace {

constexpr int kWarpKeys = 32;   // keys of a stage per consumer warp

template <int D, int HG, bool HI>
struct Q8DecCfg {
    static constexpr int kParts = 8 / HG;                 // warps per head
    static constexpr int kKeys = kWarpKeys * kParts;      // keys per stage
    static constexpr int kTileBytes = kKeys * HG * D;     // K (or V) of one stage: 32 or 16 KB
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kRows = HI ? 16 : 8;             // q rows kept per warp
    static constexpr int kMergeFloats = kParts == 1 ? 0 : 8 * kRows * (D + 2);
    static constexpr int kStages = (kParts == 1 ? 3 : 2) * (128 / D);
    static constexpr int kScaleOff = kStages * kStageBytes;       // [stage][K, V][64]: [head][block]
    static constexpr int kMergeOff = kScaleOff + kStages * 128;
    static constexpr int kBarOff = kMergeOff + 4 * kMergeFloats;
    static constexpr int kSmemBytes = kBarOff + 256 + 1024;
    static_assert(kSmemBytes <= 232448, "beyond the 227 KB of shared memory a CTA may have");
    static constexpr int kThreads = 288;
};

struct Q8DecBars {
    uint64_t full[6], empty[6];
    int abort;
};

__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The transposed 8 x 8 b16 matrix whose row g, columns 2t and 2t + 1 lane (g, t) holds.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Rows of a stage are keys: the key of index g within eight, and the column piece
// (16 bytes of 128, 8 of 64) of index g. Conflict-free for a 128-byte row whose
// chunk c sits at c ^ (row & 7), and a 64-byte row whose chunk c sits at
// c ^ (row / 2 & 3).
template <int D>
__device__ __forceinline__ int kappa(int g)
{
    const int i = g >> 1;
    return (g & 1) == 0 ? i : 4 + (D == 128 ? i : (i ^ 1));
}

template <int D>
__device__ __forceinline__ int chi(int g)
{
    return D == 128 ? ((g & 1) << 2 | g >> 1) : ((g & 1) | (g & 2) << 1 | (g & 4) >> 1);
}

// Address of 16-byte chunk c of row `row` of a tile (rows of one box and head are
// consecutive; a box starts on a multiple of eight rows).
template <int D>
__device__ __forceinline__ uint32_t chunk_addr(uint32_t base, int row, int c)
{
    return base + row * D + ((c ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4);
}

template <int D, int HG, bool HI>
__global__ void __launch_bounds__(288, 1)
decode_q8_kernel(const DecodeParams p, const Q8Cache cache, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v)
{
    using C = Q8DecCfg<D, HG, HI>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Q8DecBars *bars = reinterpret_cast<Q8DecBars *>(smem + C::kBarOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.group;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bars->full[s], 32);
            mbar_init(&bars->empty[s], 8);
        }
        bars->abort = 0;
        fence_barrier_init();
    }
    pdl_trigger();
    pdl_wait();
    const int n_items = p.counts[kCntDecode];
    __syncthreads();
    volatile int *abort = &bars->abort;
    // rows per box: within a page, and on the 64-key grid that items start on
    const int RB = min(min(p.page_size, C::kKeys), 64);
    const int lgrb = 31 - __clz(RB);
    const int lgsb = cache.lg_sb;

    if (warp == 8) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
        }
        const int NBX = C::kKeys >> lgrb;          // boxes per stage and tensor (at most 32)
        const uint32_t box_bytes = (uint32_t)HG * RB * D;
        const int blocks = C::kKeys >> lgsb;       // scale blocks per head and stage
        const int n_scales = HG * blocks;          // per tensor: 16 (SB 16) or 32 (SB 8)
        uint32_t g = 0;
        bool stop = false;
        DecodeItem w_next{};
        if (blockIdx.x < n_items)
            w_next = p.ditems[blockIdx.x];
        for (int it = blockIdx.x; it < n_items && !stop && !warp_aborted(abort); it += gridDim.x) {
            const DecodeItem w = w_next;
            if (it + (int)gridDim.x < n_items)
                w_next = p.ditems[it + gridDim.x];
            const int32_t *bt_row = p.block_table + (int64_t)w.r * p.max_blocks;
            const int head0 = w.kvh * HG;
            const int nst = (w.key1 - w.key0 + C::kKeys - 1) / C::kKeys;
            // box number b of the item (b = stage * NBX + box) and its page; lane l holds
            // boxes 32 m + l of window m, the next two windows already on their way (a stage
            // has at most 32 boxes, and scale bytes are asked for two stages ahead)
            auto lookup = [&](int m) -> int {
                const int key = w.key0 + ((32 * m + lane) << lgrb);
                return key < w.key1 ? __ldg(bt_row + (key >> cache.lg_page)) : -1;
            };
            int cur = lookup(0), nxt = lookup(1), nx2 = lookup(2);
            int window = 0;
            auto page_of = [&](int box) -> int {   // of a box in these windows (any lane asks)
                const int a = __shfl_sync(0xffffffffu, cur, box & 31), b = __shfl_sync(0xffffffffu, nxt, box & 31);
                const int c = __shfl_sync(0xffffffffu, nx2, box & 31), d = (box >> 5) - window;
                return d == 0 ? a : (d == 1 ? b : c);
            };
            // this lane's scale bytes of stage j: number lane (and lane + 32 of the 64 that
            // SB 8 has), first K's, then V's
            auto scales_of = [&](int j, uint32_t &lo, uint32_t &hi) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = lane + 32 * k;
                    uint32_t b = 0;
                    const int tensor = i >= n_scales, x = i - tensor * n_scales;
                    const int h = x / blocks, blk = x - h * blocks;
                    const int key = w.key0 + j * C::kKeys + (blk << lgsb);
                    const int pg = page_of(min(j, nst - 1) * NBX + ((blk << lgsb) >> lgrb));
                    if (i < 2 * n_scales && j < nst && key < w.key1 && pg >= 0 && pg < p.num_pages)
                        b = __ldg((tensor ? cache.vs : cache.ks) +
                                  (((int64_t)pg * p.num_kv_heads + head0 + h) << (cache.lg_page - lgsb)) +
                                  ((key & (p.page_size - 1)) >> lgsb));
                    (k == 0 ? lo : hi) = b;
                }
            };
            uint32_t s0lo, s0hi, s1lo, s1hi;
            scales_of(0, s0lo, s0hi);
            scales_of(1, s1lo, s1hi);
            for (int j = 0; j < nst; ++j, ++g) {
                const int box = j * NBX + lane;
                // the window moves on once a stage starts in the next one (NBX divides 32)
                if ((j * NBX) >> 5 != window) {
                    ++window;
                    cur = nxt;
                    nxt = nx2;
                    nx2 = lookup(window + 2);
                }
                const int pg = __shfl_sync(0xffffffffu, cur, (j * NBX + (lane & (NBX - 1))) & 31);
                uint32_t s2lo, s2hi;
                scales_of(j + 2, s2lo, s2hi);
                const int stage = g % C::kStages;
                if (g >= (uint32_t)C::kStages &&
                    !mbar_wait_warp(&bars->empty[stage], ((g / C::kStages) - 1) & 1, abort)) {
                    stop = true;
                    break;
                }
                uint8_t *kdst = smem + stage * C::kStageBytes;
                uint8_t *sc = smem + C::kScaleOff + stage * 128;
                auto put = [&](int i, uint32_t b) {
                    const int tensor = i >= n_scales;
                    if (i < 2 * n_scales)
                        sc[tensor * 64 + i - tensor * n_scales] = (uint8_t)b;
                };
                put(lane, s0lo);
                put(lane + 32, s0hi);
                // every lane arrives once, after its scale bytes; a lane with a box announces
                // that box's bytes in the same step, before it issues the copies
                const int key = w.key0 + (box << lgrb);
                const bool live = lane < NBX && key < w.key1;
                const bool valid = live && pg >= 0 && pg < p.num_pages;
                if (valid) {
                    mbar_arrive_expect_tx(&bars->full[stage], 2 * box_bytes);
                    const int off = key & (p.page_size - 1);
                    tma_load_4d(kdst + lane * box_bytes, &tm_k, &bars->full[stage], 0, off, head0, pg);
                    tma_load_4d(kdst + C::kTileBytes + lane * box_bytes, &tm_v, &bars->full[stage], 0, off, head0, pg);
                } else {
                    if (live)
                        set_dev_error(p.dev_err, CPSA_DEV_PAGE_OUT_OF_RANGE);
                    mbar_arrive(&bars->full[stage]);
                }
                s0lo = s1lo; s0hi = s1hi;
                s1lo = s2lo; s1hi = s2hi;
                __syncwarp();
            }
        }
        mbar_drain(bars->full, g, C::kStages);
        return;
    }

    // ---------------------------------------------------------------- consumers
    constexpr int NH = HI ? 2 : 1;             // n tiles of eight q heads
    constexpr int KS = D / 16;                 // k steps of a score
    constexpr int MT = D / 16;                 // m tiles of the output
    constexpr int NT = D / 8;                  // a lane's consecutive columns of the output
    const int g = lane >> 2, t = lane & 3;
    const int h = warp % HG, part = warp / HG;
    const int kb0 = part * kWarpKeys;
    uint32_t gs = 0;
    for (int it = blockIdx.x; it < n_items; it += gridDim.x) {
        const DecodeItem w = p.ditems[it];
        const int nst = (w.key1 - w.key0 + C::kKeys - 1) / C::kKeys;
        const int kvh = w.kvh * HG + h;
        // q head g (+ 8) as f16 under its own power of two; k step 4 j + x of lane t covers
        // columns 16 (t + 4 j) + 4 x + {0, 1} and {2, 3}
        uint32_t qb[KS][NH][2];
        float rf[NH][2];                       // of heads 2t, 2t + 1 (+ 8): the score's scale
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            const int row = g + 8 * nh;
            uint4 raw[KS / 2];
            float amax = 0.f;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    raw[2 * j + x] = make_uint4(0, 0, 0, 0);
                    if (row < G)
                        raw[2 * j + x] = __ldg(reinterpret_cast<const uint4 *>(
                            reinterpret_cast<const __nv_bfloat16 *>(p.q) +
                            ((int64_t)w.t * p.num_q_heads + kvh * G + row) * D + 16 * (t + 4 * j) + 8 * x));
                    amax = fmaxf(amax, bf16x8_amax(raw[2 * j + x]));
                }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const int qe = q_exponent(amax);
            const float scale = p.scale_log2 * exp2i(qe);
#pragma unroll
            for (int e = 0; e < 2; ++e) rf[nh][e] = __shfl_sync(0xffffffffu, scale, 4 * (2 * t + e));
            const float f = exp2i(-qe);
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint4 r = raw[2 * j + (x >> 1)];
                    qb[4 * j + x][nh][0] = bf16x2_to_f16x2((x & 1) ? r.z : r.x, f);
                    qb[4 * j + x][nh][1] = bf16x2_to_f16x2((x & 1) ? r.w : r.y, f);
                }
        }
        float m_run[NH][2], l_run[NH][2];
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m_run[nh][e] = -INFINITY;
                l_run[nh][e] = 0.f;
            }
        int X = -126;                          // the largest value exponent so far
        float o[MT][NH][4];
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) o[j][nh][0] = o[j][nh][1] = o[j][nh][2] = o[j][nh][3] = 0.f;

        for (int j = 0; j < nst; ++j) {
            const uint32_t gg = gs + j;
            const int stage = gg % C::kStages;
            if (!mbar_wait_warp(&bars->full[stage], (gg / C::kStages) & 1, abort))
                break;
            const int nv = w.key1 - w.key0 - j * C::kKeys - kb0;   // this warp's valid keys (may be <= 0, or > 32)
            if (nv > 0) {
                // this head's 32 rows: boxes of RB rows x HG heads; eight rows never leave a box
                const uint32_t kt = smem_u32(smem + stage * C::kStageBytes);
                auto row_base = [&](int r8) -> uint32_t {          // of the warp's rows 8 r8 .. 8 r8 + 7
                    const int key = kb0 + 8 * r8;
                    return kt + ((((key >> lgrb) * HG + h) << lgrb) + (key & (RB - 1))) * D;
                };
                // scores, keys x heads: m tile mt holds keys 16 mt .. (rows g: r8 = 2 mt, rows
                // g + 8: r8 = 2 mt + 1)
                float s[2][NH][4];
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int nh = 0; nh < NH; ++nh) s[mt][nh][0] = s[mt][nh][1] = s[mt][nh][2] = s[mt][nh][3] = 0.f;
#pragma unroll
                for (int jj = 0; jj < D / 64; ++jj) {
                    uint32_t x[4][4];
#pragma unroll
                    for (int r8 = 0; r8 < 4; ++r8) {
                        const uint4 v = lds128(chunk_addr<D>(row_base(r8), kappa<D>(g), t + 4 * jj));
                        x[r8][0] = v.x;
                        x[r8][1] = v.y;
                        x[r8][2] = v.z;
                        x[r8][3] = v.w;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt) {
                            const uint32_t a[4] = {e4m3_lo(x[2 * mt][k]), e4m3_lo(x[2 * mt + 1][k]),
                                                   e4m3_hi(x[2 * mt][k]), e4m3_hi(x[2 * mt + 1][k])};
#pragma unroll
                            for (int nh = 0; nh < NH; ++nh)
                                mma_f16(s[mt][nh], a, qb[4 * jj + k][nh][0], qb[4 * jj + k][nh][1]);
                        }
                }
                // the scale exponents of each eight keys
                const uint8_t *sc = smem + C::kScaleOff + stage * 128 + h * (C::kKeys >> lgsb) + (kb0 >> lgsb);
                float kf[4], vf[4];
                int vx[4], Xn = X;
#pragma unroll
                for (int r8 = 0; r8 < 4; ++r8) {
                    kf[r8] = exp2i(q8_exp(sc[(8 * r8) >> lgsb]));
                    vx[r8] = q8_exp(sc[64 + ((8 * r8) >> lgsb)]);
                    if (8 * r8 < nv)
                        Xn = max(Xn, vx[r8]);
                }
                const float xs = exp2i(max(X - Xn, -126));
                X = Xn;
#pragma unroll
                for (int r8 = 0; r8 < 4; ++r8) vf[r8] = exp2i(min(max(vx[r8] - X, -100), 0) + 15);
                // softmax of heads 2t, 2t + 1 (+ 8) over this lane's keys kappa(g) of each eight,
                // then over the lanes of the other g
                uint32_t pb[4][NH];
                float scale_o[NH][2];
                bool moved = false;
                const int mykey = kappa<D>(g);
#pragma unroll
                for (int nh = 0; nh < NH; ++nh) {
                    float pr[4][2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int r8 = 0; r8 < 4; ++r8) {
                            // a zero score stays zero
                            float v = s[r8 >> 1][nh][(r8 & 1) * 2 + e] * fminf(rf[nh][e] * kf[r8], 3.0e38f);
                            if (8 * r8 + mykey >= nv)
                                v = -INFINITY;
                            pr[r8][e] = v;
                            mx = fmaxf(mx, v);
                        }
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        const float m_new = fmaxf(m_run[nh][e], mx);
                        const float alpha = m_new == m_run[nh][e] ? 1.f : ex2_approx(m_run[nh][e] - m_new);
                        m_run[nh][e] = m_new;
                        const float mref = m_new == -INFINITY ? 0.f : m_new;
                        float psum = 0.f;
#pragma unroll
                        for (int r8 = 0; r8 < 4; ++r8) {
                            pr[r8][e] = ex2_approx(pr[r8][e] - mref);
                            psum += pr[r8][e];
                        }
                        l_run[nh][e] = l_run[nh][e] * alpha + psum;
                        scale_o[nh][e] = alpha * xs;
                        moved = moved || scale_o[nh][e] != 1.f;
                    }
                    // keys x heads to the heads x keys of a B operand
#pragma unroll
                    for (int r8 = 0; r8 < 4; ++r8)
                        pb[r8][nh] = transpose_8x8(pack_f16x2(pr[r8][0] * vf[r8], pr[r8][1] * vf[r8]));
                }
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int j2 = 0; j2 < MT; ++j2)
#pragma unroll
                        for (int nh = 0; nh < NH; ++nh) {
                            o[j2][nh][0] *= scale_o[nh][0];
                            o[j2][nh][1] *= scale_o[nh][1];
                            o[j2][nh][2] *= scale_o[nh][0];
                            o[j2][nh][3] *= scale_o[nh][1];
                        }
                }
                // O^T += V^T P^T, 16 keys at a time
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    constexpr int W = D / 32;              // 32-bit words of a lane's column piece
                    uint32_t rows[4][W];                   // keys kappa(2t), kappa(2t + 1) of the first and second eight
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int r8 = 2 * k + (q >> 1);
                        const int key = kappa<D>(2 * t + (q & 1));
                        const uint32_t rb = row_base(r8) + C::kTileBytes;
                        if (D == 128) {
                            const uint4 v = lds128(chunk_addr<D>(rb, key, chi<D>(g)));
                            rows[q][0] = v.x;
                            rows[q][1] = v.y;
                            rows[q][2 % W] = v.z;
                            rows[q][3 % W] = v.w;
                        } else {
                            const int piece = chi<D>(g);
                            const uint2 v = lds64(chunk_addr<D>(rb, key, piece >> 1) + (piece & 1) * 8);
                            rows[q][0] = v.x;
                            rows[q][1] = v.y;
                        }
                        if (8 * r8 + key >= nv) {          // behind the last key: may hold NaN
#pragma unroll
                            for (int x = 0; x < W; ++x) rows[q][x] = 0u;
                        }
                    }
#pragma unroll
                    for (int x = 0; x < W; ++x) {
                        const uint32_t a = __byte_perm(rows[0][x], rows[1][x], 0x5140);
                        const uint32_t b = __byte_perm(rows[0][x], rows[1][x], 0x7362);
                        const uint32_t c = __byte_perm(rows[2][x], rows[3][x], 0x5140);
                        const uint32_t d = __byte_perm(rows[2][x], rows[3][x], 0x7362);
                        const uint32_t lo[4] = {e4m3_lo(a), e4m3_hi(a), e4m3_lo(c), e4m3_hi(c)};
                        const uint32_t hi[4] = {e4m3_lo(b), e4m3_hi(b), e4m3_lo(d), e4m3_hi(d)};
#pragma unroll
                        for (int nh = 0; nh < NH; ++nh) {
                            mma_f16(o[2 * x][nh], lo, pb[2 * k][nh], pb[2 * k + 1][nh]);
                            mma_f16(o[2 * x + 1][nh], hi, pb[2 * k][nh], pb[2 * k + 1][nh]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars->empty[stage]);
        }
        gs += nst;
        // O_true = o * 2^(X - 15); lane (g, t) holds, of heads 2t + e (+ 8), the D/8 columns
        // from piece chi(g) on: column 2 j in o[j][.][e], 2 j + 1 in o[j][.][2 + e]
        const float of = exp2i(X) * exp2i(-15);
        const int col0 = chi<D>(g) * NT;
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) l_run[nh][e] += __shfl_xor_sync(0xffffffffu, l_run[nh][e], x);
        if constexpr (C::kParts == 1) {
#pragma unroll
            for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 2 * t + e + 8 * nh;
                    if (row >= G)
                        continue;
                    const int hq = kvh * G + row;
                    if (w.nsplit > 1) {
                        const int64_t pr = (int64_t)w.pbase + (int64_t)hq * w.nsplit + w.split;
#pragma unroll
                        for (int j = 0; j < MT; j += 2)
                            *reinterpret_cast<float4 *>(p.part_o + pr * D + col0 + 2 * j) =
                                make_float4(o[j][nh][e] * of, o[j][nh][2 + e] * of, o[j + 1][nh][e] * of,
                                            o[j + 1][nh][2 + e] * of);
                        if (g == 0)
                            reinterpret_cast<float2 *>(p.part_ml)[pr] = make_float2(m_run[nh][e], l_run[nh][e]);
                    } else {
                        // 1 / l and the power one after the other: their product may be no normal number
                        const float l = l_run[nh][e];
                        const float inv = l > 0.f ? 1.f / l : 0.f;   // a NaN sum leaves o NaN
                        __nv_bfloat16 *dst =
                            reinterpret_cast<__nv_bfloat16 *>(p.out) + ((int64_t)w.t * p.num_q_heads + hq) * D + col0;
#pragma unroll
                        for (int j = 0; j < MT; j += 4) {
                            uint32_t pk[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                pk[x] = pack_bf16x2(o[j + x][nh][e] * inv * of, o[j + x][nh][2 + e] * inv * of);
                            *reinterpret_cast<uint4 *>(dst + 2 * j) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                        }
                    }
                }
        } else {
            // the warps of a head meet: [warp][row] max and sum, [warp][row][D] O
            float *mm = reinterpret_cast<float *>(smem + C::kMergeOff);
            float *ll = mm + 8 * C::kRows;
            float *oo = ll + 8 * C::kRows;
#pragma unroll
            for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 2 * t + e + 8 * nh;
                    if (row >= G)
                        continue;
                    if (g == 0) {
                        mm[warp * C::kRows + row] = m_run[nh][e];
                        ll[warp * C::kRows + row] = l_run[nh][e];
                    }
                    float *dst = oo + (warp * C::kRows + row) * D + col0;
#pragma unroll
                    for (int j = 0; j < MT; j += 2)
                        *reinterpret_cast<float4 *>(dst + 2 * j) =
                            make_float4(o[j][nh][e] * of, o[j][nh][2 + e] * of, o[j + 1][nh][e] * of,
                                        o[j + 1][nh][2 + e] * of);
                }
            named_bar_sync(1, 256);
            for (int e = threadIdx.x; e < HG * G * D; e += 256) {
                const int hh = e / (G * D), row = e / D % G, d = e % D;
                float M = -INFINITY;
#pragma unroll
                for (int x = 0; x < C::kParts; ++x) M = fmaxf(M, mm[(x * HG + hh) * C::kRows + row]);
                const float Mref = M == -INFINITY ? 0.f : M;
                float L = 0.f, acc = 0.f;
#pragma unroll
                for (int x = 0; x < C::kParts; ++x) {
                    const int at = (x * HG + hh) * C::kRows + row;
                    const float f = ex2_approx(mm[at] - Mref);
                    L += f * ll[at];
                    acc += f * oo[at * D + d];
                }
                const int hq = (w.kvh * HG + hh) * G + row;
                if (w.nsplit > 1) {
                    const int64_t pr = (int64_t)w.pbase + (int64_t)hq * w.nsplit + w.split;
                    p.part_o[pr * D + d] = acc;
                    if (d == 0)
                        reinterpret_cast<float2 *>(p.part_ml)[pr] = make_float2(M, L);
                } else {
                    reinterpret_cast<__nv_bfloat16 *>(p.out)[((int64_t)w.t * p.num_q_heads + hq) * D + d] =
                        __float2bfloat16_rn(acc * (L > 0.f ? 1.f / L : 0.f));
                }
            }
            named_bar_sync(1, 256);
        }
    }
    if (threadIdx.x == 0 && *abort)
        set_dev_error(p.dev_err, CPSA_DEV_WAIT_TIMEOUT);
}

template <int D, int HG, bool HI>
cudaError_t launch_t(const DecodeParams &p, const Q8Cache &c, const CUtensorMap &tk, const CUtensorMap &tv, int grid,
                     cudaStream_t s, bool early)
{
    using C = Q8DecCfg<D, HG, HI>;
    static std::atomic<uint64_t> done{0};
    auto k = decode_q8_kernel<D, HG, HI>;
    return launch_with_smem(done, reinterpret_cast<const void *>(k), C::kSmemBytes, [&] {
        return launch_pdl(early, k, dim3(grid), dim3(C::kThreads), C::kSmemBytes, s, p, c, tk, tv);
    });
}

template <int D, int HG>
cudaError_t launch_hg(const DecodeParams &p, const Q8Cache &c, const CUtensorMap &tk, const CUtensorMap &tv, int grid,
                      cudaStream_t s, bool early)
{
    return p.group > 8 ? launch_t<D, HG, true>(p, c, tk, tv, grid, s, early)
                       : launch_t<D, HG, false>(p, c, tk, tv, grid, s, early);
}

template <int D>
cudaError_t launch_d(const DecodeParams &p, const Q8Cache &c, const CUtensorMap &tk, const CUtensorMap &tv, int heads,
                     int grid, cudaStream_t s, bool early)
{
    switch (heads) {
    case 8: return launch_hg<D, 8>(p, c, tk, tv, grid, s, early);
    case 4: return launch_hg<D, 4>(p, c, tk, tv, grid, s, early);
    case 2: return launch_hg<D, 2>(p, c, tk, tv, grid, s, early);
    default: return launch_hg<D, 1>(p, c, tk, tv, grid, s, early);
    }
}

}  // namespace

cudaError_t launch_decode_q8(const DecodeParams &p, const Q8Cache &c, const CUtensorMap &tk, const CUtensorMap &tv,
                             int head_dim, int heads_per_item, int grid, cudaStream_t s, bool early)
{
    return head_dim == 128 ? launch_d<128>(p, c, tk, tv, heads_per_item, grid, s, early)
                           : launch_d<64>(p, c, tk, tv, heads_per_item, grid, s, early);
}

// Rows per TMA box of the decode kernel (abi.cu builds the maps with it).
int decode_q8_box_rows(int page_size, int heads_per_item)
{
    const int keys = kWarpKeys * (8 / heads_per_item);
    const int rows = page_size < keys ? page_size : keys;
    return rows < 64 ? rows : 64;
}

}  // namespace cpsa
