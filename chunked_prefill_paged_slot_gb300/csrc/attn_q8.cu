// attn_q8.cu -- causal attention over the 8-bit paged cache (e4m3 bytes, one
// power-of-two scale per block of SB places and kv head; the format is
// rope_append.cu's). Same masks, metadata and device flags as the bf16 kernels.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.cuh"
#include "plan.cuh"

namespace cpsa {

namespace {

// 2^(b - 127) (0 and 255, which the writer never stores, as their neighbours)
__device__ __forceinline__ float q8_scale(uint8_t b)
{
    return __uint_as_float((uint32_t)(b < 1 ? 1 : (b > 254 ? 254 : b)) << 23);
}

// Four bytes as fp32.
__device__ __forceinline__ void q8_widen4(uint32_t w, float (&f)[4])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w >> (16 * i))));
        const float2 x = __half22float2(*reinterpret_cast<__half2 *>(&h));
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
    }
}

constexpr int kPlainWarps = 8;

// Chunks (query_len >= 2): one CTA per (new token, q head); warp w takes every eighth key, a lane D/32
// columns; the warps' (max, sum, O) meet in shared memory.
template <int D>
__global__ void __launch_bounds__(32 * kPlainWarps)
attn_q8_row_kernel(const AttnCommon p, const Q8Cache c, const __nv_bfloat16 *q, int num_reqs, int num_tokens)
{
    constexpr int CPL = D / 32;
    __shared__ float sm[kPlainWarps], sl[kPlainWarps], so[kPlainWarps][D];
    const int t = blockIdx.x, h = blockIdx.y, kvh = h / p.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    if (p.counts[kCntPrefill] + p.counts[kCntDecode] == 0)   // nothing to do, or the plan refused the batch
        return;
    int lo = 0, hi = num_reqs - 1;   // the last request that starts at or before t (its rows hold t)
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu_q[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int r = lo, s = p.seq_lens[r], ql = p.query_lens[r];
    if (ql < 2 || t < p.cu_q[r] || t - p.cu_q[r] >= ql || s < ql || (int64_t)s > (int64_t)p.max_blocks * p.page_size)
        return;
    const int last = s - ql + (t - p.cu_q[r]);
    float qv[CPL], o[CPL], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < CPL; ++e) {
        qv[e] = __bfloat162float(q[((int64_t)t * p.num_q_heads + h) * D + lane * CPL + e]) * p.scale_log2;
        o[e] = 0.f;
    }
    for (int j = warp; j <= last; j += kPlainWarps) {
        const int page = p.block_table[(int64_t)r * p.max_blocks + (j >> c.lg_page)];
        if (page < 0 || page >= p.num_pages) {
            set_dev_error(p.dev_err, CPSA_DEV_PAGE_OUT_OF_RANGE);
            continue;
        }
        const int off = j & (p.page_size - 1);
        const int64_t ph = (int64_t)page * p.num_kv_heads + kvh;
        const int64_t row = (ph * p.page_size + off) * D + lane * CPL;
        const int64_t blk = ph * (p.page_size >> c.lg_sb) + (off >> c.lg_sb);
        float kf[4], vf[4];
        q8_widen4(CPL == 4 ? *reinterpret_cast<const uint32_t *>(c.k + row)
                           : *reinterpret_cast<const uint16_t *>(c.k + row), kf);
        q8_widen4(CPL == 4 ? *reinterpret_cast<const uint32_t *>(c.v + row)
                           : *reinterpret_cast<const uint16_t *>(c.v + row), vf);
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < CPL; ++e) x = fmaf(qv[e], kf[e], x);
        for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
        x *= q8_scale(c.ks[blk]);
        const float mn = fmaxf(m, x);
        const float a = mn == m ? 1.f : ex2_approx(m - mn), pj = ex2_approx(x - mn);
        const float pv = pj * q8_scale(c.vs[blk]);
        m = mn;
        l = l * a + pj;
#pragma unroll
        for (int e = 0; e < CPL; ++e) o[e] = fmaf(pv, vf[e], o[e] * a);
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < CPL; ++e) so[warp][lane * CPL + e] = o[e];
    __syncthreads();
    if (threadIdx.x < D) {
        float M = -INFINITY, L = 0.f, acc = 0.f;
        for (int w = 0; w < kPlainWarps; ++w) M = fmaxf(M, sm[w]);
        const float ref = M == -INFINITY ? 0.f : M;
        for (int w = 0; w < kPlainWarps; ++w) {
            const float f = ex2_approx(sm[w] - ref);
            L += f * sl[w];
            acc += f * so[w][threadIdx.x];
        }
        reinterpret_cast<__nv_bfloat16 *>(p.out)[((int64_t)t * p.num_q_heads + h) * D + threadIdx.x] =
            __float2bfloat16_rn(acc * (L > 0.f ? 1.f / L : 0.f));   // a NaN sum leaves acc NaN
    }
}

}  // namespace

cudaError_t launch_attn_q8_rows(const AttnCommon &p, const Q8Cache &c, const void *q, int head_dim, int num_reqs,
                                int num_tokens, cudaStream_t s, bool early)
{
    const dim3 grid(num_tokens, p.num_q_heads);
    if (head_dim == 128)
        return launch_pdl(early, attn_q8_row_kernel<128>, grid, dim3(32 * kPlainWarps), 0, s, p, c,
                          (const __nv_bfloat16 *)q, num_reqs, num_tokens);
    return launch_pdl(early, attn_q8_row_kernel<64>, grid, dim3(32 * kPlainWarps), 0, s, p, c,
                      (const __nv_bfloat16 *)q, num_reqs, num_tokens);
}

}  // namespace cpsa
