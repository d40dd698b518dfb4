// idx_latent_prefill.cu -- expanded latent attention of ragged sequences:
// s = scale * (q[:128] . k + q[128:] . k_rope), out = softmax(s) . v.
//
// One warp per (query, head): a lane scores one key of 32, the warp folds the
// 32 into its running maximum and sum, and each lane keeps four of the 128
// output elements.
#include <cuda_bf16.h>

#include "idx_common.cuh"
#include "idx_internal.h"

namespace idx {
namespace {

constexpr int kThreads = 128;
constexpr int kNope = 128, kRope = 64, kV = 128, kQk = kNope + kRope;

struct PrefillArgs {
    const __nv_bfloat16 *q, *k, *k_rope, *v;
    int64_t ldq_row, ldq_head, ldk_row, ldk_head, ld_rope, ldv_row, ldv_head;
    const int32_t *cu_q, *cu_k;
    int B, Tq, Tk, H;
    float scale;
    int causal;
    __nv_bfloat16 *out;
    int64_t ldo_row, ldo_head;
    float *lse;
    int64_t ld_lse;
};

__global__ void __launch_bounds__(kThreads) latent_prefill_kernel(PrefillArgs a)
{
    __shared__ float qs[kThreads / 32][kQk];
    pdl_wait();
    const int w = threadIdx.x >> 5, lane = lane_id(), h = blockIdx.y;
    const int row = blockIdx.x * (kThreads / 32) + w;
    const int total = min(a.Tq, a.cu_q[a.B]);
    if (row >= total || row < a.cu_q[0])
        return;
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.cu_q[mid] <= row)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int nq = min(a.cu_q[lo + 1], total) - a.cu_q[lo];
    const int k0 = a.cu_k[lo], nk = min(a.cu_k[lo + 1], a.Tk) - k0;
    const int end = a.causal ? min(nk, row - a.cu_q[lo] + nk - nq + 1) : nk;
    for (int d = lane; d < kQk; d += 32)
        qs[w][d] = __bfloat162float(a.q[row * a.ldq_row + h * a.ldq_head + d]);
    __syncwarp();
    float m = -INFINITY, l = 0.0f, acc[4] = {};
    for (int j0 = 0; j0 < end; j0 += 32) {
        const int j = j0 + lane;
        float s = -INFINITY;
        if (j < end) {
            const __nv_bfloat16 *k = a.k + (k0 + j) * a.ldk_row + h * a.ldk_head;
            const __nv_bfloat16 *kr = a.k_rope + (k0 + j) * a.ld_rope;
            s = 0.0f;
            for (int d = 0; d < kNope; ++d)
                s = fmaf(qs[w][d], __bfloat162float(k[d]), s);
            for (int d = 0; d < kRope; ++d)
                s = fmaf(qs[w][kNope + d], __bfloat162float(kr[d]), s);
            s *= a.scale;
        }
        float nm = fmaxf(m, s);
        #pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, o));
        const float c = __expf(m - nm), p = __expf(s - nm);
        float ps = p;
        #pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            ps += __shfl_xor_sync(0xffffffffu, ps, o);
        l = l * c + ps;
        m = nm;
        #pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[i] *= c;
        const int cnt = min(32, end - j0);
        for (int t = 0; t < cnt; ++t) {
            const float pt = __shfl_sync(0xffffffffu, p, t);
            const __nv_bfloat16 *v = a.v + (k0 + j0 + t) * a.ldv_row + h * a.ldv_head;
            #pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i] = fmaf(pt, __bfloat162float(v[32 * i + lane]), acc[i]);
        }
    }
    #pragma unroll
    for (int i = 0; i < 4; ++i)
        a.out[row * a.ldo_row + h * a.ldo_head + 32 * i + lane] =
            __float2bfloat16(l == 0.0f ? 0.0f : acc[i] / l);
    if (a.lse && lane == 0)
        a.lse[row * a.ld_lse + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

} // namespace
} // namespace idx

using namespace idx;

extern "C" idx_status idx_latent_prefill(const uint16_t *q, int64_t ldq_row, int64_t ldq_head,
                                         const uint16_t *k, int64_t ldk_row, int64_t ldk_head,
                                         const uint16_t *k_rope, int64_t ld_rope,
                                         const uint16_t *v, int64_t ldv_row, int64_t ldv_head,
                                         const int32_t *cu_q, const int32_t *cu_k, int B, int Tq,
                                         int Tk, int H, int d_nope, int d_rope, int d_v,
                                         float scale, int causal, uint16_t *out, int64_t ldo_row,
                                         int64_t ldo_head, float *lse, int64_t ld_lse,
                                         idx_stream_t stream)
{
    IDX_NVTX_RANGE("idx_latent_prefill");
    if (B < 0 || Tq < 0 || Tk < 0 || H <= 0 || d_nope <= 0 || d_rope < 0 || d_v <= 0)
        return IDX_ERR_INVALID_ARG;
    if (B == 0 || Tq == 0)
        return IDX_OK;
    if (!q || !cu_q || !cu_k || !out || (Tk > 0 && (!k || !k_rope || !v)) || !(scale > 0.0f) ||
        !(scale <= 3.4e38f) || ldq_head < (int64_t)d_nope + d_rope || ldq_row < 0 ||
        ldk_head < d_nope || ldk_row < 0 || ld_rope < d_rope || ldv_head < d_v || ldv_row < 0 ||
        ldo_head < d_v || ldo_row < 0 || (lse && ld_lse < H))
        return IDX_ERR_INVALID_ARG;
    if (d_nope != kNope || d_rope != kRope || d_v != kV || H > 65535 || !aligned16(q) ||
        !aligned16(k) || !aligned16(k_rope) || !aligned16(v) || !aligned16(out) ||
        (ldq_row | ldq_head | ldk_row | ldk_head | ld_rope | ldv_row | ldv_head | ldo_row |
         ldo_head) % 8 != 0)
        return IDX_ERR_UNSUPPORTED;
    const auto bf = [](const uint16_t *p) { return reinterpret_cast<const __nv_bfloat16 *>(p); };
    PrefillArgs a = {bf(q), bf(k), bf(k_rope), bf(v), ldq_row, ldq_head, ldk_row, ldk_head,
                     ld_rope, ldv_row, ldv_head, cu_q, cu_k, B, Tq, Tk, H, scale, causal,
                     reinterpret_cast<__nv_bfloat16 *>(out), ldo_row, ldo_head, lse, ld_lse};
    return launch_status(launch_pdl(latent_prefill_kernel,
                                    dim3((Tq + kThreads / 32 - 1) / (kThreads / 32), H),
                                    dim3(kThreads), 0, (cudaStream_t)stream, a));
}
