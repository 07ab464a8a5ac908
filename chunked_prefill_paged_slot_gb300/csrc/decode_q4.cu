// decode_q4.cu -- split-KV attention of decode rows (query_len == 1) over the 4-bit
// paged cache (q4.cuh): every byte of the row's context is read once, for all the q
// heads of its kv head at once.
//
// softmax(scale * q K^T) V over keys [key0, key1) of one row, for HG kv heads (8, 4,
// 2 or 1 by what divides the head count) and their G q heads each.
//
// CTA (288 threads, persistent over the plan's items):
//   warp 8     producer: stages of 8 WK / HG keys of HG heads; per page (or 64 rows of
//              one) one TMA box each of K's and V's codes and scales, covering the heads;
//              page numbers a window of stages ahead.
//   warps 0..7 warp w: kv head w % HG of the group, keys [WK (w / HG), + WK) of every
//              stage. The 8 / HG warps of a head meet in shared memory at the end.
//
// Arithmetic. A number of the cache is exact in f16, so operands are made by one cvt
// and one f16 multiplication per two numbers; of q, each row is brought to f16 by a power
// of two that puts its largest element in [2^14, 2^15) (what that drops is under 2^-39 of
// the row's largest). The running maximum is only raised where a stage exceeds it by more
// than 2^8, so most stages spend one vote on it and no shuffles; probabilities are at most
// 2^8 under it and enter f16 times 2^7 (the sum with them, so O / l stays), whole down to
// 2^-21 of the maximum. Sums in fp32.
//
// Keys are the M rows of the scores (mma.sync m16n8k16: 16 keys x 16 columns times 16
// columns x 8 heads), columns those of the output (16 columns x 16 keys times 16 keys x 8
// heads). Fragments are chosen for the loads, the k index of an mma being a free
// relabelling: lane (g, t) = (lane / 4, lane % 4) takes, of key kappa(g) of each eight, the
// quarter t of the row (one load, whole groups); of V, for the keys kappa(2t), kappa(2t + 1)
// of each eight, the eighth chi(g) of the row, the two keys' codes brought into (key, key)
// bytes by shifts and masks before they are converted. kappa and chi are such that the
// loads of a warp are free of bank conflicts.
//
// Measured (32/8 heads, D 128, pages of 16): 384 rows of 1024 to 8192 keys, 2.1 GB, 334 us
// replayed in a graph, 6.3 TB/s or 94 % of a plain copy's rate, and 334 to 344 us a call. That is
// with the plan, an empty chunk launch and the combine; with the arithmetic skipped a call took
// 338 us where it took 350 (by an earlier plan), so what is left is loading and those three. Not kept: 16 warps on half stages (407 us),
// the scores of one stage beside the output of the one before (402 us).
#include "common.cuh"
#include "kernels.cuh"
#include "plan.cuh"
#include "q4.cuh"
#include "q8.cuh"

namespace cpsa {

namespace {

constexpr int kP2 = 7;   // probabilities are held times 2^kP2

// ROWS: q heads per kv head that a warp has room for: 4, 8 or 16.
template <int D, int HG, int ROWS>
struct Q4DecCfg {
    static constexpr int kParts = 8 / HG;                 // warps per head
    static constexpr int kRow = D / 2, kScRow = D / kQ4Group;   // bytes of a row's codes and scales
    static constexpr int kMergeFloats = kParts == 1 ? 0 : 4 * ROWS * (D + 2);
    // keys of a stage per warp: 64 (384 rows of 1024 to 8192 keys, 32/8 heads: 371 us, 401 us at 32);
    // 32 where a stage would have over 32 boxes, the scores of 16 heads would spill, or only two
    // stages would fit beside the merge
    static constexpr int WK = HG == 1 || ROWS == 16 || (D == 128 && kParts > 1 && ROWS > 4) ? 32 : 64;
    static constexpr int kKeys = WK * kParts;             // keys per stage
    static constexpr int kTileBytes = kKeys * HG * kRow;  // codes of K (or V) of one stage
    static constexpr int kScTile = 4096;                  // its scales, in boxes of at least 128 bytes
    static constexpr int kStageBytes = 2 * (kTileBytes + kScTile);
    static constexpr int kRoom = (232448 - 1024 - 256 - 4 * kMergeFloats) / kStageBytes;
    static constexpr int kStages = kRoom < 6 ? kRoom : 6;
    static constexpr int kMergeOff = kStages * kStageBytes;
    static constexpr int kBarOff = kMergeOff + 4 * kMergeFloats;
    static constexpr int kSmemBytes = kBarOff + 256 + 1024;
    static_assert(kSmemBytes <= 232448 && kStages >= 3, "beyond the 227 KB of shared memory a CTA may have");
    static_assert(kKeys * HG * kScRow <= kScTile, "a stage's scales");
    static constexpr int kThreads = 288;
};

struct Q4DecBars {
    uint64_t full[6], empty[6];
    int abort;
};

__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ uint32_t lds8(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
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

// The key of index g within eight, and the eighth of a row of index g. Rows of 64 bytes
// (D 128) have their 16-byte chunk c at c ^ (row / 2 & 3); K's quarter is such a chunk, V's
// eighth half of one. Rows of 32 bytes (D 64) lie as they are: eight lanes' quarters or the
// four rows of a V load cover all banks where their rows differ modulo 4.
template <int D>
__device__ __forceinline__ int kappa(int g)
{
    if (D == 128) {
        const int i = g >> 1;
        return (g & 1) == 0 ? i : 4 + (i ^ 1);
    }
    return (0x67453210 >> (4 * g)) & 7;   // 0 1 2 3 5 4 7 6
}

template <int D>
__device__ __forceinline__ int chi(int g)
{
    return D == 128 ? ((g & 1) | (g & 2) << 1 | (g & 4) >> 1) : g;
}

// The items of a batch of one decode row: the plan's (plan.cu: decode_splits, request_work).
struct OneRow {
    int s, splits, items;   // keys; splits; items (0: nothing to do)
    __device__ __forceinline__ DecodeItem item(int k, int ngroups) const
    {
        const int sp = k / ngroups, tiles = (s + kDecodeChunk - 1) / kDecodeChunk;
        const int c0 = sp * tiles / splits, c1 = (sp + 1) * tiles / splits;
        return DecodeItem{0, k - sp * ngroups, c0 * kDecodeChunk, min(c1 * kDecodeChunk, s), sp, splits,
                          splits > 1 ? 0 : -1, 0};
    }
};

// The row's checks and splits; CTA 0 reports, and leaves the combine kernel its list.
template <int HG>
__device__ __forceinline__ OneRow one_row(const DecodeParams &p)
{
    const int q = __ldg(p.query_lens), s = __ldg(p.seq_lens);
    uint32_t bad = 0;
    if (q != 1)
        bad = CPSA_DEV_TOKENS_MISMATCH;
    else if (s < 1)
        bad = CPSA_DEV_SEQ_LT_QUERY;
    else if (!fits_table(s, p.max_blocks, p.page_size))
        bad = CPSA_DEV_SEQ_GT_TABLE;
    OneRow row{s, 1, 0};
    if (!bad) {
        row.splits = max(1, min(min((s + p.dec_keys - 1) / p.dec_keys, p.max_splits), (s + kDecodeChunk - 1) / kDecodeChunk));
        row.items = row.splits * (p.num_kv_heads / HG);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (bad || p.split_clamped)
            set_dev_error(p.dev_err, bad | (p.split_clamped ? CPSA_DEV_SPLITS_CLAMPED : 0u));
        const bool merge = row.splits > 1;
        if (merge)
            p.citems_w[0] = CombineItem{0, 1, 0, p.num_q_heads, 0, row.splits, 0, 0};
        p.counts_w[kCntCombine] = merge ? 1 : 0;
        p.counts_w[kCntCombineUnits] = merge ? p.num_q_heads : 0;
    }
    return row;
}

template <int D, int HG, int ROWS>
__global__ void __launch_bounds__(288, 1)
decode_q4_kernel(const DecodeParams p, const Q4Cache cache, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_ks,
                 const __grid_constant__ CUtensorMap tm_vs)
{
    using C = Q4DecCfg<D, HG, ROWS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Q4DecBars *bars = reinterpret_cast<Q4DecBars *>(smem + C::kBarOff);
    // (one value a warp, which keeps the arithmetic on it off the lanes)
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
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
    // this CTA's items: a run of the plan's list, or every gridDim.x-th of it or of the row's own
    const bool runs = p.run_first != nullptr;
    const OneRow row = p.self_plan ? one_row<HG>(p) : OneRow{0, 0, 0};
    const int it_begin = runs ? p.run_first[blockIdx.x] : blockIdx.x;
    const int it_end = p.self_plan ? row.items : runs ? p.run_first[blockIdx.x + 1] : p.counts[kCntDecode];
    const int it_step = runs ? 1 : gridDim.x;
    auto item = [&](int it) -> DecodeItem { return p.self_plan ? row.item(it, p.num_kv_heads / HG) : p.ditems[it]; };
    __syncthreads();
    volatile int *abort = &bars->abort;
    // rows per box: within a page, and on the 64-key grid that items start on
    const int RB = min(min(p.page_size, C::kKeys), 64);
    const int lgrb = 31 - __clz(RB);
    const int sc_pitch = max(128, HG * RB * C::kScRow);   // a scale box (its address: a multiple of 128)

    if (warp == 8) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
            tma_prefetch_desc(&tm_ks);
            tma_prefetch_desc(&tm_vs);
        }
        const int NBX = C::kKeys >> lgrb;          // boxes per stage and tensor (at most 32)
        const uint32_t box_bytes = (uint32_t)HG * RB * C::kRow, sc_bytes = (uint32_t)HG * RB * C::kScRow;
        uint32_t g = 0;
        bool stop = false;
        DecodeItem w_next{};
        if (it_begin < it_end)
            w_next = item(it_begin);
        for (int it = it_begin; it < it_end && !stop && !warp_aborted(abort); it += it_step) {
            const DecodeItem w = w_next;
            if (it + it_step < it_end)
                w_next = item(it + it_step);
            const int32_t *bt_row = p.block_table + (int64_t)w.r * p.max_blocks;
            const int head0 = w.kvh * HG;
            const int nst = (w.key1 - w.key0 + C::kKeys - 1) / C::kKeys;
            // box number b of the item (b = stage * NBX + box) and its page; lane l holds
            // boxes 32 m + l of window m, the next window's already on its way
            auto lookup = [&](int m) -> int {
                const int key = w.key0 + ((32 * m + lane) << lgrb);
                return key < w.key1 ? ldg_here(bt_row + (key >> cache.lg_page)) : -1;
            };
            int cur = lookup(0), nxt = lookup(1);
            int window = 0;
            for (int j = 0; j < nst; ++j, ++g) {
                const int box = j * NBX + lane;
                // the window moves on once a stage starts in the next one (NBX divides 32)
                if ((j * NBX) >> 5 != window) {
                    ++window;
                    cur = nxt;
                    nxt = lookup(window + 1);
                }
                int pg = __shfl_sync(0xffffffffu, cur, (j * NBX + (lane & (NBX - 1))) & 31);
                const int stage = g % C::kStages;
                if (g >= (uint32_t)C::kStages &&
                    !mbar_wait_warp(&bars->empty[stage], ((g / C::kStages) - 1) & 1, abort)) {
                    stop = true;
                    break;
                }
                uint8_t *kdst = smem + stage * C::kStageBytes;
                uint8_t *sdst = kdst + 2 * C::kTileBytes + lane * sc_pitch;
                // every lane arrives once; a lane with a box announces that box's bytes in the
                // same step, before it issues the copies
                const int key = w.key0 + (box << lgrb);
                const bool live = lane < NBX && key < w.key1;
                if (live) {
                    if (pg < 0 || pg >= p.num_pages) {
                        set_dev_error(p.dev_err, CPSA_DEV_PAGE_OUT_OF_RANGE);
                        pg = -1;   // a box ahead of the cache's first: the copies bring zeros
                    }
                    mbar_arrive_expect_tx(&bars->full[stage], 2 * (box_bytes + sc_bytes));
                    const int off = key & (p.page_size - 1);
                    const int sc_off = off * (C::kScRow / 4);   // in words
                    tma_load_4d(kdst + lane * box_bytes, &tm_k, &bars->full[stage], 0, off, head0, pg);
                    tma_load_3d(sdst, &tm_ks, &bars->full[stage], sc_off, head0, pg);
                    tma_load_4d(kdst + C::kTileBytes + lane * box_bytes, &tm_v, &bars->full[stage], 0, off, head0, pg);
                    tma_load_3d(sdst + C::kScTile, &tm_vs, &bars->full[stage], sc_off, head0, pg);
                } else {
                    mbar_arrive(&bars->full[stage]);
                }
                __syncwarp();
            }
        }
        mbar_drain(bars->full, g, C::kStages);
        return;
    }

    // ---------------------------------------------------------------- consumers
    constexpr int NH = ROWS == 16 ? 2 : 1;             // n tiles of eight q heads
    constexpr int KS = D / 16;                 // k steps of a score
    constexpr int MT = D / 16;                 // m tiles of the output
    constexpr int R8 = C::WK / 8;              // eights of a warp's keys
    constexpr int KW = D / 32;                 // words of a K quarter
    constexpr int VW = D / 64;                 // words of a V eighth
    const int g = lane >> 2, t = lane & 3;
    const int h = warp % HG, part = warp / HG;
    const int kb0 = part * C::WK;
    const int kkey = kappa<D>(g), vkey0 = kappa<D>(2 * t), vkey1 = kappa<D>(2 * t + 1), vpiece = chi<D>(g);
    // byte offsets of this lane's pieces within eight rows
    const uint32_t k_off = D == 128 ? kkey * 64 + ((t ^ (kkey >> 1 & 3)) << 4) : kkey * 32 + t * 8;
    auto v_off = [&](int key) -> uint32_t {
        return D == 128 ? key * 64 + (((vpiece >> 1) ^ (key >> 1 & 3)) << 4) + (vpiece & 1) * 8 : key * 32 + vpiece * 4;
    };
    const uint32_t v_off0 = v_off(vkey0), v_off1 = v_off(vkey1);
    const uint32_t ks_off = kkey * C::kScRow + t * (D / 64);
    const uint32_t vs_piece = D == 128 ? vpiece : vpiece >> 1;
    const uint32_t vs_off0 = vkey0 * C::kScRow + vs_piece, vs_off1 = vkey1 * C::kScRow + vs_piece;
    uint32_t gs = 0;
    for (int it = it_begin; it < it_end; it += it_step) {
        const DecodeItem w = item(it);
        const int nst = (w.key1 - w.key0 + C::kKeys - 1) / C::kKeys;
        const int kvh = w.kvh * HG + h;
        // q head g (+ 8) as f16 under its own power of two; k step s of lane t covers
        // columns (D / 4) t + 4 s + {0, 1} and {2, 3}
        uint32_t qb[KS][NH][2];
        float rf[NH][2];                       // of heads 2t, 2t + 1 (+ 8): the score's scale
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            const int row = g + 8 * nh;
            uint4 raw[KS / 2];
            float amax = 0.f;
#pragma unroll
            for (int x = 0; x < KS / 2; ++x) {
                raw[x] = make_uint4(0, 0, 0, 0);
                if (row < G)
                    raw[x] = __ldg(reinterpret_cast<const uint4 *>(
                        reinterpret_cast<const __nv_bfloat16 *>(p.q) +
                        ((int64_t)w.t * p.num_q_heads + kvh * G + row) * D + (D / 4) * t + 8 * x));
                amax = fmaxf(amax, bf16x8_amax(raw[x]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const int qe = q_exponent(amax);
            // never 0 or infinite: a masked score times it stays -inf, a zero one 0
            const float scale = fminf(fmaxf(p.scale_log2 * exp2i(qe), 1.2e-38f), 3.0e38f);
#pragma unroll
            for (int e = 0; e < 2; ++e) rf[nh][e] = __shfl_sync(0xffffffffu, scale, 4 * (2 * t + e));
            const float f = exp2i(-qe);
#pragma unroll
            for (int x = 0; x < KS / 2; ++x) {
                qb[2 * x][nh][0] = bf16x2_to_f16x2(raw[x].x, f);
                qb[2 * x][nh][1] = bf16x2_to_f16x2(raw[x].y, f);
                qb[2 * x + 1][nh][0] = bf16x2_to_f16x2(raw[x].z, f);
                qb[2 * x + 1][nh][1] = bf16x2_to_f16x2(raw[x].w, f);
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
            const int nv = w.key1 - w.key0 - j * C::kKeys - kb0;   // this warp's valid keys (may be <= 0, or > WK)
            if (nv > 0) {
                // this head's rows: boxes of RB rows x HG heads; eight rows never leave a box
                const uint32_t kt = smem_u32(smem + stage * C::kStageBytes);
                uint32_t row8[R8], sc8[R8];
#pragma unroll
                for (int r8 = 0; r8 < R8; ++r8) {
                    const int key = kb0 + 8 * r8, box = key >> lgrb, off = key & (RB - 1);
                    row8[r8] = kt + (((box * HG + h) << lgrb) + off) * C::kRow;
                    sc8[r8] = kt + 2 * C::kTileBytes + box * sc_pitch + ((h << lgrb) + off) * C::kScRow;
                }
                // scores, keys x heads: m tile mt holds keys 16 mt .. (rows g: r8 = 2 mt, rows
                // g + 8: r8 = 2 mt + 1)
                float s[R8 / 2][NH][4];
#pragma unroll
                for (int mt = 0; mt < R8 / 2; ++mt)
#pragma unroll
                    for (int nh = 0; nh < NH; ++nh) s[mt][nh][0] = s[mt][nh][1] = s[mt][nh][2] = s[mt][nh][3] = 0.f;
                // the m tiles in turn, so that no mma waits for the one right before it
                uint32_t x[R8][KW], sc[R8];
#pragma unroll
                for (int r8 = 0; r8 < R8; ++r8) {
                    if (D == 128) {
                        const uint4 v = lds128(row8[r8] + k_off);
                        x[r8][0] = v.x;
                        x[r8][1] = v.y;
                        x[r8][2 % KW] = v.z;
                        x[r8][3 % KW] = v.w;
                        sc[r8] = lds_u16(sc8[r8] + ks_off);
                    } else {
                        const uint2 v = lds64(row8[r8] + k_off);
                        x[r8][0] = v.x;
                        x[r8][1] = v.y;
                        sc[r8] = lds8(sc8[r8] + ks_off);
                    }
                }
#pragma unroll
                for (int k = 0; k < KW; ++k)
#pragma unroll
                    for (int mt = 0; mt < R8 / 2; ++mt) {
                        uint32_t f[2][4];
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const uint32_t sf = q4_scale2(k < 2 ? sc[2 * mt + b] & 0xffu : sc[2 * mt + b] >> 8);
                            e2m1x8(x[2 * mt + b][k], f[b]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) f[b][i] = q4_mul(f[b][i], sf);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t a[4] = {f[0][2 * i], f[1][2 * i], f[0][2 * i + 1], f[1][2 * i + 1]};
#pragma unroll
                            for (int nh = 0; nh < NH; ++nh)
                                mma_f16(s[mt][nh], a, qb[2 * k + i][nh][0], qb[2 * k + i][nh][1]);
                        }
                    }
                // keys behind the last one
                if (nv < C::WK) {
#pragma unroll
                    for (int r8 = 0; r8 < R8; ++r8)
                        if (8 * r8 + kkey >= nv)
#pragma unroll
                            for (int nh = 0; nh < NH; ++nh)
                                s[r8 >> 1][nh][(r8 & 1) * 2] = s[r8 >> 1][nh][(r8 & 1) * 2 + 1] = -INFINITY;
                }
                // heads 2t + e (+ 8): this lane's largest scores; where one is far above the
                // running maximum, all maxima are raised to the warp's
                float mx[NH][2];
                bool need = false;
#pragma unroll
                for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = -INFINITY;
#pragma unroll
                        for (int r8 = 0; r8 < R8; r8 += 2) m = fmax3(m, s[r8 >> 1][nh][e], s[r8 >> 1][nh][2 + e]);
                        mx[nh][e] = m * rf[nh][e];
                        need = need || mx[nh][e] > m_run[nh][e] + 8.f;
                    }
                if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                    for (int nh = 0; nh < NH; ++nh) {
                        float alpha[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float m = mx[nh][e];
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                            m = fmaxf(m, m_run[nh][e]);
                            alpha[e] = m == m_run[nh][e] ? 1.f : ex2_approx(m_run[nh][e] - m);
                            m_run[nh][e] = m;
                            l_run[nh][e] *= alpha[e];
                        }
#pragma unroll
                        for (int j2 = 0; j2 < MT; ++j2) {
                            o[j2][nh][0] *= alpha[0];
                            o[j2][nh][1] *= alpha[1];
                            o[j2][nh][2] *= alpha[0];
                            o[j2][nh][3] *= alpha[1];
                        }
                    }
                }
                // probabilities, keys x heads to the heads x keys of a B operand
                uint32_t pb[R8][NH];
#pragma unroll
                for (int nh = 0; nh < NH; ++nh) {
                    float ref[2], sum[2] = {0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < 2; ++e) ref[e] = (float)kP2 - (m_run[nh][e] == -INFINITY ? 0.f : m_run[nh][e]);
#pragma unroll
                    for (int r8 = 0; r8 < R8; ++r8) {
                        const float a = ex2_approx(fmaf(s[r8 >> 1][nh][(r8 & 1) * 2], rf[nh][0], ref[0]));
                        const float b = ex2_approx(fmaf(s[r8 >> 1][nh][(r8 & 1) * 2 + 1], rf[nh][1], ref[1]));
                        sum[0] += a;
                        sum[1] += b;
                        pb[r8][nh] = transpose_8x8(pack_f16x2(a, b));
                    }
                    l_run[nh][0] += sum[0];
                    l_run[nh][1] += sum[1];
                }
                // O^T += V^T P^T, 16 keys at a time
#pragma unroll
                for (int k = 0; k < R8 / 2; ++k) {
                    uint32_t v[2][2][VW], sp[2];       // [eight][key 2t, 2t + 1]; their scales as a pair
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const uint32_t rb = row8[2 * k + b] + C::kTileBytes, sb = sc8[2 * k + b] + C::kScTile;
                        uint32_t s0 = lds8(sb + vs_off0), s1 = lds8(sb + vs_off1);
                        if (D == 128) {
                            const uint2 a = lds64(rb + v_off0), c = lds64(rb + v_off1);
                            v[b][0][0] = a.x;
                            v[b][0][1 % VW] = a.y;
                            v[b][1][0] = c.x;
                            v[b][1][1 % VW] = c.y;
                        } else {
                            v[b][0][0] = lds32(rb + v_off0);
                            v[b][1][0] = lds32(rb + v_off1);
                        }
                        if (nv < C::WK) {              // behind the last key: may hold NaN
                            if (8 * (2 * k + b) + vkey0 >= nv)
                                s0 = 0;
                            if (8 * (2 * k + b) + vkey1 >= nv)
                                s1 = 0;
                        }
                        sp[b] = (s0 | s1 << 16) << 7;
                    }
#pragma unroll
                    for (int x = 0; x < VW; ++x) {
                        // bytes of (key, key) codes: even columns, odd columns
                        uint32_t ev[2][4], od[2][4];
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const uint32_t a = v[b][0][x], c = v[b][1][x];
                            e2m1x8((a & 0x0f0f0f0fu) | ((c << 4) & 0xf0f0f0f0u), ev[b]);
                            e2m1x8(((a >> 4) & 0x0f0f0f0fu) | (c & 0xf0f0f0f0u), od[b]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                ev[b][i] = q4_mul(ev[b][i], sp[b]);
                                od[b][i] = q4_mul(od[b][i], sp[b]);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t a[4] = {ev[0][i], od[0][i], ev[1][i], od[1][i]};
#pragma unroll
                            for (int nh = 0; nh < NH; ++nh)
                                mma_f16(o[4 * x + i][nh], a, pb[2 * k][nh], pb[2 * k + 1][nh]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars->empty[stage]);
        }
        gs += nst;
        // lane (g, t) holds, of heads 2t + e (+ 8), the D/8 columns from piece chi(g) on: column
        // 2 j in o[j][.][e], 2 j + 1 in o[j][.][2 + e]
        const int col0 = vpiece * (D / 8);
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) l_run[nh][e] += __shfl_xor_sync(0xffffffffu, l_run[nh][e], x);
        if constexpr (C::kParts > 1) {
            // the warps of a head meet by halves: the upper ones leave their maximum, sum and O in
            // shared memory, the lower ones take them in, until one is left
            float *mm = reinterpret_cast<float *>(smem + C::kMergeOff);
            float *ll = mm + 4 * ROWS;
            float *oo = ll + 4 * ROWS;
#pragma unroll
            for (int half = C::kParts / 2; half >= 1; half /= 2) {
                const int at = (part % half) * HG + h;      // of a pair of warps
                if (part >= half && part < 2 * half) {
#pragma unroll
                    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int row = 2 * t + e + 8 * nh;
                            if (row >= G)
                                continue;
                            if (g == 0) {
                                mm[at * ROWS + row] = m_run[nh][e];
                                ll[at * ROWS + row] = l_run[nh][e];
                            }
                            float *dst = oo + (at * ROWS + row) * D + col0;
#pragma unroll
                            for (int j = 0; j < MT; j += 2)
                                *reinterpret_cast<float4 *>(dst + 2 * j) =
                                    make_float4(o[j][nh][e], o[j][nh][2 + e], o[j + 1][nh][e], o[j + 1][nh][2 + e]);
                        }
                }
                named_bar_sync(1, 256);
                if (part < half) {
#pragma unroll
                    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int row = 2 * t + e + 8 * nh;
                            if (row >= G)
                                continue;
                            const float m2 = mm[at * ROWS + row], M = fmaxf(m_run[nh][e], m2);
                            const float Mref = M == -INFINITY ? 0.f : M;
                            const float f1 = ex2_approx(m_run[nh][e] - Mref), f2 = ex2_approx(m2 - Mref);
                            m_run[nh][e] = M;
                            l_run[nh][e] = f1 * l_run[nh][e] + f2 * ll[at * ROWS + row];
                            const float *src = oo + (at * ROWS + row) * D + col0;
#pragma unroll
                            for (int j = 0; j < MT; j += 2) {
                                const float4 x = *reinterpret_cast<const float4 *>(src + 2 * j);
                                o[j][nh][e] = f1 * o[j][nh][e] + f2 * x.x;
                                o[j][nh][2 + e] = f1 * o[j][nh][2 + e] + f2 * x.y;
                                o[j + 1][nh][e] = f1 * o[j + 1][nh][e] + f2 * x.z;
                                o[j + 1][nh][2 + e] = f1 * o[j + 1][nh][2 + e] + f2 * x.w;
                            }
                        }
                }
                named_bar_sync(1, 256);
            }
        }
        if (part == 0) {
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
                                make_float4(o[j][nh][e], o[j][nh][2 + e], o[j + 1][nh][e], o[j + 1][nh][2 + e]);
                        if (g == 0)
                            reinterpret_cast<float2 *>(p.part_ml)[pr] = make_float2(m_run[nh][e], l_run[nh][e]);
                    } else {
                        const float l = l_run[nh][e];
                        const float inv = l > 0.f ? 1.f / l : 0.f;   // a NaN sum leaves o NaN
                        __nv_bfloat16 *dst =
                            reinterpret_cast<__nv_bfloat16 *>(p.out) + ((int64_t)w.t * p.num_q_heads + hq) * D + col0;
#pragma unroll
                        for (int j = 0; j < MT; j += 4) {
                            uint32_t pk[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                pk[x] = pack_bf16x2(o[j + x][nh][e] * inv, o[j + x][nh][2 + e] * inv);
                            *reinterpret_cast<uint4 *>(dst + 2 * j) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                        }
                    }
                }
        }
    }
    if (threadIdx.x == 0 && *abort)
        set_dev_error(p.dev_err, CPSA_DEV_WAIT_TIMEOUT);
}

template <int D, int HG, int ROWS>
cudaError_t launch_t(const DecodeParams &p, const Q4Cache &c, const Q4Maps &m, int grid, cudaStream_t s, bool early)
{
    using C = Q4DecCfg<D, HG, ROWS>;
    static std::atomic<uint64_t> done{0};
    auto k = decode_q4_kernel<D, HG, ROWS>;
    return launch_with_smem(done, reinterpret_cast<const void *>(k), C::kSmemBytes, [&] {
        return launch_pdl(early, k, dim3(grid), dim3(C::kThreads), C::kSmemBytes, s, p, c, m.k, m.v, m.ks, m.vs);
    });
}

template <int D, int HG>
cudaError_t launch_hg(const DecodeParams &p, const Q4Cache &c, const Q4Maps &m, int grid, cudaStream_t s, bool early)
{
    if (p.group > 8)
        return launch_t<D, HG, 16>(p, c, m, grid, s, early);
    // all of a page's heads to a warp each: nothing to merge, and no room to keep for it
    return p.group > 4 || HG == 8 ? launch_t<D, HG, 8>(p, c, m, grid, s, early)
                                  : launch_t<D, HG, HG == 8 ? 8 : 4>(p, c, m, grid, s, early);
}

template <int D>
cudaError_t launch_d(const DecodeParams &p, const Q4Cache &c, const Q4Maps &m, int heads, int grid, cudaStream_t s,
                     bool early)
{
    switch (heads) {
    case 8: return launch_hg<D, 8>(p, c, m, grid, s, early);
    case 4: return launch_hg<D, 4>(p, c, m, grid, s, early);
    case 2: return launch_hg<D, 2>(p, c, m, grid, s, early);
    default: return launch_hg<D, 1>(p, c, m, grid, s, early);
    }
}

template <int D, int HG>
int stage_keys(int group)
{
    return group > 8   ? Q4DecCfg<D, HG, 16>::kKeys
           : group > 4 ? Q4DecCfg<D, HG, 8>::kKeys
                       : Q4DecCfg<D, HG, HG == 8 ? 8 : 4>::kKeys;
}

template <int D>
int stage_keys(int heads, int group)
{
    return heads == 8   ? stage_keys<D, 8>(group)
           : heads == 4 ? stage_keys<D, 4>(group)
           : heads == 2 ? stage_keys<D, 2>(group)
                        : stage_keys<D, 1>(group);
}

}  // namespace

cudaError_t launch_decode_q4(const DecodeParams &p, const Q4Cache &c, const Q4Maps &m, int head_dim,
                             int heads_per_item, int grid, cudaStream_t s, bool early)
{
    return head_dim == 128 ? launch_d<128>(p, c, m, heads_per_item, grid, s, early)
                           : launch_d<64>(p, c, m, heads_per_item, grid, s, early);
}

// Rows per TMA box of the decode kernel (abi.cu builds the maps with it).
int decode_q4_box_rows(int head_dim, int page_size, int heads_per_item, int group)
{
    const int keys = head_dim == 128 ? stage_keys<128>(heads_per_item, group) : stage_keys<64>(heads_per_item, group);
    const int rows = page_size < keys ? page_size : keys;
    return rows < 64 ? rows : 64;
}

}  // namespace cpsa
