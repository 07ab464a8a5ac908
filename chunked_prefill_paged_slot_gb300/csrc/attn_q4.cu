// attn_q4.cu -- causal attention over the 4-bit paged cache (q4.cuh). Same masks, metadata and
// device flags as the bf16 kernels. One CTA per (new token, q head): warp w takes every eighth
// key, a lane D/32 columns; the warps' (max, sum, O) meet in shared memory.
#include "common.cuh"
#include "kernels.cuh"
#include "plan.cuh"
#include "q4.cuh"

namespace cpsa {

namespace {

constexpr int kRowWarps = 8;

// CPL columns of one group (a byte or two of codes) as fp32.
template <int CPL>
__device__ __forceinline__ void widen(uint32_t codes, uint32_t scale_byte, float (&f)[CPL])
{
    uint32_t h[4];
    e2m1x8(codes, h);
    const float s = __half2float(__ushort_as_half((unsigned short)(scale_byte << 7)));
#pragma unroll
    for (int i = 0; i < CPL / 2; ++i) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        f[2 * i] = x.x * s;
        f[2 * i + 1] = x.y * s;
    }
}

template <int D>
__global__ void __launch_bounds__(32 * kRowWarps)
attn_q4_row_kernel(const AttnCommon p, const Q4Cache c, const __nv_bfloat16 *q, int num_reqs)
{
    constexpr int CPL = D / 32;
    __shared__ float sm[kRowWarps], sl[kRowWarps], so[kRowWarps][D];
    const int t = blockIdx.x, h = blockIdx.y, kvh = h / p.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    if (p.counts[kCntPrefill] + p.counts[kCntDecode] == 0)   // nothing to do, or the plan refused the batch
        return;
    int lo = 0, hi = num_reqs - 1;   // the last request that starts at or before t (its rows hold t)
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu_q[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int r = lo, s = p.seq_lens[r], ql = p.query_lens[r];
    if (t < p.cu_q[r] || t - p.cu_q[r] >= ql || s < ql || (int64_t)s > (int64_t)p.max_blocks * p.page_size)
        return;
    const int last = s - ql + (t - p.cu_q[r]);
    float qv[CPL], o[CPL], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < CPL; ++e) {
        qv[e] = __bfloat162float(q[((int64_t)t * p.num_q_heads + h) * D + lane * CPL + e]) * p.scale_log2;
        o[e] = 0.f;
    }
    for (int j = warp; j <= last; j += kRowWarps) {
        const int page = p.block_table[(int64_t)r * p.max_blocks + (j >> c.lg_page)];
        if (page < 0 || page >= p.num_pages) {
            set_dev_error(p.dev_err, CPSA_DEV_PAGE_OUT_OF_RANGE);
            continue;
        }
        const int64_t row = ((((int64_t)page * p.num_kv_heads + kvh) << c.lg_page) + (j & (p.page_size - 1)));
        const int64_t at = row * (D / 2) + lane * (CPL / 2), sc = row * (D / kQ4Group) + lane * CPL / kQ4Group;
        float kf[CPL], vf[CPL];
        widen<CPL>(CPL == 4 ? *reinterpret_cast<const uint16_t *>(c.k + at) : c.k[at], c.ks[sc], kf);
        widen<CPL>(CPL == 4 ? *reinterpret_cast<const uint16_t *>(c.v + at) : c.v[at], c.vs[sc], vf);
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < CPL; ++e) x = fmaf(qv[e], kf[e], x);
        for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
        const float mn = fmaxf(m, x);
        const float a = mn == m ? 1.f : ex2_approx(m - mn), pj = ex2_approx(x - mn);
        m = mn;
        l = l * a + pj;
#pragma unroll
        for (int e = 0; e < CPL; ++e) o[e] = fmaf(pj, vf[e], o[e] * a);
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
        for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, sm[w]);
        const float ref = M == -INFINITY ? 0.f : M;
        for (int w = 0; w < kRowWarps; ++w) {
            const float f = ex2_approx(sm[w] - ref);
            L += f * sl[w];
            acc += f * so[w][threadIdx.x];
        }
        reinterpret_cast<__nv_bfloat16 *>(p.out)[((int64_t)t * p.num_q_heads + h) * D + threadIdx.x] =
            __float2bfloat16_rn(acc * (L > 0.f ? 1.f / L : 0.f));   // a NaN sum leaves acc NaN
    }
}

}  // namespace

cudaError_t launch_attn_q4_rows(const AttnCommon &p, const Q4Cache &c, const void *q, int head_dim, int num_reqs,
                                int num_tokens, cudaStream_t s, bool early)
{
    const dim3 grid(num_tokens, p.num_q_heads);
    return launch_pdl(early, head_dim == 128 ? attn_q4_row_kernel<128> : attn_q4_row_kernel<64>, grid,
                      dim3(32 * kRowWarps), 0, s, p, c, static_cast<const __nv_bfloat16 *>(q), num_reqs);
}

}  // namespace cpsa
