// idx_latent_attn.cu -- absorbed latent attention over ragged slots or whole
// paged contexts:  s = scale * q . token,  out = softmax(s) . token[:512].
//
// One CTA per (row, eight heads), a warp per head; tokens are decoded into
// shared memory sixteen at a time and folded into a running maximum, sum and
// 512 accumulators (sixteen a lane).
#include <cuda_fp8.h>

#include "idx_latent.cuh"

namespace idx {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 16;

struct AttnArgs {
    LatentPool pool;
    int fp8;
    const uint16_t *q;
    int64_t ldq_row, ldq_head;
    const int32_t *slots, *indptr;  // sparse
    int64_t num_slots;
    const int32_t *block_table, *context_lens;  // paged
    int64_t bt_stride;
    int ctx_per_row, next_n, max_len;
    int R, H;
    float scale;
    uint16_t *out;
    int64_t ldo_row, ldo_head;
    float *lse;
    int64_t ld_lse;
    unsigned int *status;
};

__global__ void __launch_bounds__(kThreads) latent_attn_kernel(AttnArgs a)
{
    __shared__ float tok[kTile][kLatTok];
    __shared__ int good[kTile];
    pdl_wait();
    const int r = blockIdx.x, lane = lane_id(), h = blockIdx.y * 8 + (threadIdx.x >> 5);
    const bool live = h < a.H;
    int64_t first = 0;
    int n;
    if (a.indptr) {
        const int64_t lo = min((int64_t)max(a.indptr[r], 0), a.num_slots);
        const int64_t hi = min((int64_t)max(a.indptr[r + 1], 0), a.num_slots);
        first = lo;
        n = (int)max((int64_t)0, hi - lo);
    } else {
        const int b = r / a.next_n, j = r % a.next_n;
        const int end = a.ctx_per_row ? a.context_lens[r] : a.context_lens[b] - a.next_n + j + 1;
        n = min(max(end, 0), a.max_len);
    }
    float q[18], acc[16] = {}, m = -INFINITY, l = 0.0f;
    #pragma unroll
    for (int i = 0; i < 18; ++i)
        q[i] = live ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(
                          a.q)[r * a.ldq_row + h * a.ldq_head + 32 * i + lane])
                    : 0.0f;
    for (int t0 = 0; t0 < n; t0 += kTile) {
        __syncthreads();
        for (int e = threadIdx.x; e < kTile * kLatTok; e += kThreads) {
            const int k = e / kLatTok, d = e % kLatTok, t = t0 + k;
            float v = 0.0f;
            bool ok = false;
            if (t < n) {
                int64_t slot;
                if (a.indptr) {
                    slot = a.slots[first + t];
                } else {
                    const int p = page_of(a.pool, t);
                    const int id = a.block_table[(int64_t)(r / a.next_n) * a.bt_stride + p];
                    slot = id < 0 ? -1 : (int64_t)id * a.pool.page_size + (t - p * a.pool.page_size);
                }
                int64_t pb;
                int off;
                ok = slot_place(a.pool, slot, &pb, &off);
                if (!ok) {
                    if (d == 0)
                        atomicOr(a.status, kDevBadPage);
                } else if (!a.fp8) {
                    v = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(
                        a.pool.base + pb + (int64_t)off * kLatBf16TokBytes)[d]);
                } else if (d < kLatent) {
                    __nv_fp8_e4m3 c;
                    c.__x = a.pool.base[pb + (int64_t)off * kLatent + d];
                    const int s = a.pool.base[pb + (int64_t)a.pool.page_size * 640 +
                                              (int64_t)off * kLatGroups + d / kLatGroup];
                    v = s == 255 ? NAN : ldexpf((float)c, s - 127);
                    v = __bfloat162float(__float2bfloat16(v));
                } else {
                    v = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(
                        a.pool.base + pb + (int64_t)a.pool.page_size * kLatent +
                        (int64_t)off * 2 * kLatRope)[d - kLatent]);
                }
            }
            tok[k][d] = v;
            if (d == 0)
                good[k] = ok;
        }
        __syncthreads();
        for (int k = 0; k < kTile; ++k) {
            if (!good[k])
                continue;
            float s = 0.0f;
            #pragma unroll
            for (int i = 0; i < 18; ++i)
                s = fmaf(q[i], tok[k][32 * i + lane], s);
            #pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, o);
            s *= a.scale;
            const float nm = fmaxf(m, s), c = __expf(m - nm), p = __expf(s - nm);
            l = l * c + p;
            m = nm;
            #pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[i] = acc[i] * c + p * tok[k][32 * i + lane];
        }
    }
    if (!live)
        return;
    #pragma unroll
    for (int i = 0; i < 16; ++i)
        reinterpret_cast<__nv_bfloat16 *>(a.out)[r * a.ldo_row + h * a.ldo_head + 32 * i + lane] =
            __float2bfloat16(l == 0.0f ? 0.0f : acc[i] / l);
    if (a.lse && lane == 0)
        a.lse[r * a.ld_lse + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

idx_status check_attn(const uint16_t *q, int64_t ldq_row, int64_t ldq_head, int R, int H, int L,
                      int rope_dim, float scale, const uint16_t *out, int64_t ldo_row,
                      int64_t ldo_head, const float *lse, int64_t ld_lse)
{
    if (!q || !out || ldq_head < (int64_t)L + rope_dim || ldq_row < 0 || ldo_head < L ||
        ldo_row < 0 || !(scale > 0.0f) || !(scale <= 3.4e38f) || (lse && ld_lse < H))
        return IDX_ERR_INVALID_ARG;
    if (L != kLatent || rope_dim != kLatRope || H > 128 || !aligned16(q) || !aligned16(out) ||
        ldq_row % 8 != 0 || ldq_head % 8 != 0 || ldo_row % 8 != 0 || ldo_head % 8 != 0)
        return IDX_ERR_UNSUPPORTED;
    return IDX_OK;
}

idx_status run_attn(AttnArgs &a, void *ws, size_t ws_bytes, cudaStream_t s)
{
    if (!ws || ws_bytes < idx_latent_attention_workspace_size(a.R, a.H))
        return IDX_ERR_WORKSPACE;
    a.status = device_status_ptr();
    if (!a.status)
        return IDX_ERR_CUDA;
    return launch_status(launch_pdl(latent_attn_kernel, dim3(a.R, (a.H + 7) / 8), dim3(kThreads), 0,
                                    s, a));
}

} // namespace
} // namespace idx

using namespace idx;

extern "C" size_t idx_latent_attention_workspace_size(int R, int H)
{
    return R > 0 && H > 0 ? 16 : 0;
}

extern "C" idx_status idx_latent_attention(
    const uint16_t *q, int64_t ldq_row, int64_t ldq_head, const uint8_t *kv_pages,
    int64_t page_stride_bytes, int num_pages, int page_size, idx_latent_format fmt,
    const int32_t *slots, const int32_t *indptr, int64_t num_slots, int R, int H, int L,
    int rope_dim, float scale, uint16_t *out, int64_t ldo_row, int64_t ldo_head, float *lse,
    int64_t ld_lse, void *ws, size_t ws_bytes, idx_stream_t stream)
{
    IDX_NVTX_RANGE("idx_latent_attention");
    if (R < 0 || H <= 0 || L <= 0 || rope_dim < 0 || num_slots < 0)
        return IDX_ERR_INVALID_ARG;
    if (R == 0)
        return IDX_OK;
    if (!indptr || (num_slots > 0 && !slots))
        return IDX_ERR_INVALID_ARG;
    idx_status ok = check_attn(q, ldq_row, ldq_head, R, H, L, rope_dim, scale, out, ldo_row,
                               ldo_head, lse, ld_lse);
    if (ok == IDX_OK)
        ok = check_pool(kv_pages, page_stride_bytes, num_pages, page_size, fmt);
    if (ok != IDX_OK)
        return ok;
    AttnArgs a = {};
    a.pool = make_pool(kv_pages, page_stride_bytes, num_pages, page_size);
    a.fp8 = fmt == IDX_LATENT_FP8_E4M3;
    a.q = q;
    a.ldq_row = ldq_row;
    a.ldq_head = ldq_head;
    a.slots = slots;
    a.indptr = indptr;
    a.num_slots = num_slots;
    a.next_n = 1;
    a.R = R;
    a.H = H;
    a.scale = scale;
    a.out = out;
    a.ldo_row = ldo_row;
    a.ldo_head = ldo_head;
    a.lse = lse;
    a.ld_lse = ld_lse;
    return run_attn(a, ws, ws_bytes, (cudaStream_t)stream);
}

extern "C" idx_status idx_paged_latent_attention(
    const uint16_t *q, int64_t ldq_row, int64_t ldq_head, const uint8_t *kv_pages,
    int64_t page_stride_bytes, int num_pages, int page_size, idx_latent_format fmt,
    const int32_t *block_table, int64_t bt_stride, const int32_t *context_lens, int ctx_per_row,
    int B, int next_n, int max_model_len, int H, int L, int rope_dim, float scale, uint16_t *out,
    int64_t ldo_row, int64_t ldo_head, float *lse, int64_t ld_lse, void *ws, size_t ws_bytes,
    idx_stream_t stream)
{
    IDX_NVTX_RANGE("idx_paged_latent_attention");
    if (B < 0 || next_n <= 0 || max_model_len < 0 || H <= 0 || L <= 0 || rope_dim < 0 ||
        (int64_t)B * next_n > INT32_MAX)
        return IDX_ERR_INVALID_ARG;
    if (B == 0)
        return IDX_OK;
    idx_status ok = check_attn(q, ldq_row, ldq_head, B * next_n, H, L, rope_dim, scale, out,
                               ldo_row, ldo_head, lse, ld_lse);
    if (ok == IDX_OK)
        ok = check_pool(kv_pages, page_stride_bytes, num_pages, page_size, fmt);
    if (ok != IDX_OK)
        return ok;
    if (!context_lens || (max_model_len > 0 && !block_table) ||
        bt_stride < ((int64_t)max_model_len + page_size - 1) / page_size)
        return IDX_ERR_INVALID_ARG;
    AttnArgs a = {};
    a.pool = make_pool(kv_pages, page_stride_bytes, num_pages, page_size);
    a.fp8 = fmt == IDX_LATENT_FP8_E4M3;
    a.q = q;
    a.ldq_row = ldq_row;
    a.ldq_head = ldq_head;
    a.block_table = block_table;
    a.bt_stride = bt_stride;
    a.context_lens = context_lens;
    a.ctx_per_row = ctx_per_row;
    a.next_n = next_n;
    a.max_len = max_model_len;
    a.R = B * next_n;
    a.H = H;
    a.scale = scale;
    a.out = out;
    a.ldo_row = ldo_row;
    a.ldo_head = ldo_head;
    a.lse = lse;
    a.ld_lse = ld_lse;
    return run_attn(a, ws, ws_bytes, (cudaStream_t)stream);
}
