// idx_latent_cache.cu -- writer and read-back of the paged latent cache.
//
// Store: y = x / sqrt(mean(x^2) + eps) * w over a token's 512 latents, a
// rotation of its 64 positional elements by the token's angles, and for the
// 8-bit pages one power-of-two scale per 64 latents (a power of two so that
// the attention kernels can undo it exactly in bf16).  Read-back: the inverse
// look-up, slot by slot, into contiguous rows.
//
// Both move about 2 KB a token and compute next to nothing, so they are bound
// by latency (decode steps) or bandwidth (prompts, contexts): one warp holds a
// token (the norm and the group maxima are then shuffles), and every load of
// the token is issued before any is used.  Measured: 256 tokens stored 2.1 us
// (either format), 8192 tokens 4.8 us in 8 bits and 4.6 in bf16; 131072 8-bit
// tokens read back 39.4 us, 6.0 TB/s (0.88 of a copy's rate); 10007 bf16 tokens
// of five sequences 4.8 us.
#include <cuda_fp8.h>

#include "idx_latent.cuh"

namespace idx {
namespace {

constexpr int kCacheThreads = 128;
constexpr unsigned kDevBadPosition = 8u;

__device__ __forceinline__ float lo_float(uint32_t b)
{
    return __uint_as_float(b << 16);
}

__device__ __forceinline__ float hi_float(uint32_t b)
{
    return __uint_as_float(b & 0xffff0000u);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The smallest biased exponent whose power of two brings amax to 448 =
// 1.75 * 2^8 or below, read off amax's bits; 255 (e8m0 NaN) if amax is not
// finite.
__device__ __forceinline__ int group_bits(float amax)
{
    if (!(amax <= 3.4028234e38f))
        return 255;
    const uint32_t u = __float_as_uint(fmaxf(amax, 1.17549435e-38f));
    const int bits = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(bits, 0);
}

// 2^(127 - bits); 0 keeps the codes of a NaN group defined.
__device__ __forceinline__ float group_inverse(int bits)
{
    return bits == 255 ? 0.0f : __uint_as_float((uint32_t)(254 - bits) << 23);
}

// Of a token's latents, sixteen a lane.
__device__ __forceinline__ float sum_of_squares(const float (&y)[16])
{
    float ss = 0.0f;
    #pragma unroll
    for (int i = 0; i < 16; ++i)
        ss = fmaf(y[i], y[i], ss);
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    return ss;
}

// Lane l holds latents 8 l .. 8 l + 7 of both halves of 256 (16-byte loads,
// 512 contiguous bytes a warp), so a group of 64 is eight lanes, and the pair
// 2 l, 2 l + 1 of the rotated elements.
template <bool FP8>
__global__ void __launch_bounds__(kCacheThreads)
    latent_store_kernel(const uint16_t *__restrict__ kv, int64_t ld_kv,
                        const int32_t *__restrict__ positions, const float *__restrict__ cos_sin,
                        int64_t ld_cs, int num_pos, const float *__restrict__ norm_w, float eps,
                        int T, LatentPool pool, const int64_t *__restrict__ slots,
                        unsigned int *status)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = lane_id();
    const int warps = gridDim.x * (kCacheThreads / 32);
    for (int t = blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5); t < T; t += warps) {
        const int64_t slot = slots[t];
        const int pos = cos_sin ? positions[t] : 0;
        const uint16_t *row = kv + (int64_t)t * ld_kv;
        const uint4 raw[2] = {*reinterpret_cast<const uint4 *>(row + 8 * lane),
                              *reinterpret_cast<const uint4 *>(row + 256 + 8 * lane)};
        const uint32_t rope = *reinterpret_cast<const uint32_t *>(row + kLatent + 2 * lane);
        if (slot < 0)
            continue;
        const bool in_pool = slot < (int64_t)pool.num_pages * pool.page_size;
        const int page_id = in_pool ? page_of(pool, (int)slot) : 0;
        const int off = (int)slot - page_id * pool.page_size;
        const int64_t page_byte = page_id * pool.stride;
        const bool in_table = !cos_sin || (pos >= 0 && pos < num_pos);
        if (!in_pool || !in_table) {
            if (lane == 0)
                atomicOr(status, (in_pool ? 0u : kDevBadPage) | (in_table ? 0u : kDevBadPosition));
            continue;
        }
        float c = 1.0f, s = 0.0f;
        if (cos_sin) {
            const float *cs = cos_sin + (int64_t)pos * ld_cs;
            c = cs[lane];
            s = cs[kLatRope / 2 + lane];
        }
        float y[16];
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w[4] = {raw[h].x, raw[h].y, raw[h].z, raw[h].w};
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[8 * h + 2 * i] = lo_float(w[i]);
                y[8 * h + 2 * i + 1] = hi_float(w[i]);
            }
        }
        if (norm_w) {
            float ss = sum_of_squares(y), e = eps;
            if (!(ss <= 1e36f) || (ss < 1e-30f && eps < 1e-30f)) {
                // squares leave 32 bits' range: x / sqrt(mean(x^2) + eps) is the
                // same of 2^k x and 2^2k eps (uniform in the warp)
                const float up = ss < 1.0f ? 0x1p80f : 0x1p-80f;
                #pragma unroll
                for (int i = 0; i < 16; ++i)
                    y[i] *= up;
                ss = sum_of_squares(y);
                e = eps * up * up;
            }
            const float r = 1.0f / sqrtf(ss * (1.0f / kLatent) + e);
            #pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 w = *reinterpret_cast<const float4 *>(norm_w + (q >> 1) * 256 +
                                                                   8 * lane + 4 * (q & 1));
                y[4 * q] = y[4 * q] * r * w.x;
                y[4 * q + 1] = y[4 * q + 1] * r * w.y;
                y[4 * q + 2] = y[4 * q + 2] * r * w.z;
                y[4 * q + 3] = y[4 * q + 3] * r * w.w;
            }
        }
        const float a = lo_float(rope), b = hi_float(rope);
        const uint32_t turned = pack_bf16(a * c - b * s, b * c + a * s);
        uint8_t *page = const_cast<uint8_t *>(pool.base) + page_byte;
        if constexpr (!FP8) {
            uint8_t *tok = page + (int64_t)off * kLatBf16TokBytes;
            #pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<uint4 *>(tok + 512 * h + 16 * lane) =
                    make_uint4(pack_bf16(y[8 * h], y[8 * h + 1]),
                               pack_bf16(y[8 * h + 2], y[8 * h + 3]),
                               pack_bf16(y[8 * h + 4], y[8 * h + 5]),
                               pack_bf16(y[8 * h + 6], y[8 * h + 7]));
            *reinterpret_cast<uint32_t *>(tok + 2 * kLatent + 4 * lane) = turned;
        } else {
            int bits[2];
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                float amax = 0.0f;
                bool bad = false;
                #pragma unroll
                for (int i = 0; i < 8; ++i) {
                    amax = fmaxf(amax, fabsf(y[8 * h + i]));
                    bad |= y[8 * h + i] != y[8 * h + i];  // fmaxf drops a NaN
                }
                amax = bad ? __int_as_float(0x7f800000) : amax;
                #pragma unroll
                for (int o = 1; o < 8; o <<= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                bits[h] = group_bits(amax);
                const float inv = group_inverse(bits[h]);
                uint32_t code[2];
                #pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float *v = y + 8 * h + 4 * q;
                    const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2(v[0] * inv, v[1] * inv),
                                                                __NV_SATFINITE, __NV_E4M3);
                    const uint32_t u = __nv_cvt_float2_to_fp8x2(make_float2(v[2] * inv, v[3] * inv),
                                                                __NV_SATFINITE, __NV_E4M3);
                    code[q] = l | u << 16;
                }
                *reinterpret_cast<uint2 *>(page + (int64_t)off * kLatent + 256 * h + 8 * lane) =
                    make_uint2(code[0], code[1]);
            }
            *reinterpret_cast<uint32_t *>(page + (int64_t)pool.page_size * kLatent +
                                          (int64_t)off * 2 * kLatRope + 4 * lane) = turned;
            uint8_t *scales = page + (int64_t)pool.page_size * (kLatent + 2 * kLatRope) +
                              (int64_t)off * kLatGroups;
            if ((lane & 7) == 0) {
                scales[lane >> 3] = (uint8_t)bits[0];
                scales[4 + (lane >> 3)] = (uint8_t)bits[1];
            }
        }
    }
}

// Four e4m3 codes times a power of two, as bf16.  The product is exact in
// fp32 and rounds only outside bf16's range.
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w, float scale)
{
    float2 f[2];
    #pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
        f[i] = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    }
    return make_uint2(pack_bf16(f[0].x * scale, f[0].y * scale),
                      pack_bf16(f[1].x * scale, f[1].y * scale));
}

// 2^(bits - 127), NaN for 255.
__device__ __forceinline__ float e8m0_float(uint32_t bits)
{
    return bits == 255 ? __uint_as_float(0x7fc00000u)
                       : (bits ? __uint_as_float(bits << 23) : __uint_as_float(0x400000u));
}

// A warp reads four consecutive output rows at a time: their look-ups run in
// four lanes at once, and their loads (2.6 or 4.6 KB) are in flight together.
constexpr int kGatherRows = 4;

template <bool FP8>
__global__ void __launch_bounds__(kCacheThreads)
    latent_gather_kernel(LatentPool pool, const int32_t *__restrict__ block_table,
                         int64_t bt_stride, int max_blocks, const int32_t *__restrict__ cu_lens,
                         const int32_t *__restrict__ seq_starts, int B, int N,
                         uint16_t *__restrict__ out, int64_t ld_out, unsigned int *status)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = lane_id();
    const long long step = (long long)gridDim.x * (kCacheThreads / 32) * kGatherRows;
    const int rows = cu_lens[B], total = min(N, rows);
    if (rows > N && blockIdx.x == 0 && threadIdx.x == 0)
        atomicOr(status, kDevBadBounds);
    for (long long first = ((long long)blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5)) *
                           kGatherRows;
         first < total; first += step) {
        // lanes 0..3: the row's sequence (the last b with cu_lens[b] <= row),
        // its page and its offset; -1 for a token outside the table or pool
        int64_t place = -1;
        int off = 0;
        const long long row = first + lane;
        if (lane < kGatherRows && row < total) {
            int lo = 0, hi = B - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu_lens[mid] <= row)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int64_t t = row - cu_lens[lo] + (seq_starts ? seq_starts[lo] : 0);
            const int64_t col = t < 0 ? -1 : t / pool.page_size;
            off = (int)(t - col * pool.page_size);
            const int id = col >= 0 && col < max_blocks
                               ? block_table[(int64_t)lo * bt_stride + col]
                               : -1;
            if (id >= 0 && id < pool.num_pages)
                place = (int64_t)id * pool.stride;
            else
                atomicOr(status, kDevBadPage);
        }
        int64_t at[kGatherRows];
        int o[kGatherRows];
        #pragma unroll
        for (int r = 0; r < kGatherRows; ++r) {
            at[r] = __shfl_sync(0xffffffffu, place, r);
            o[r] = __shfl_sync(0xffffffffu, off, r);
        }
        const int live = (int)min((long long)kGatherRows, total - first);
        if (FP8) {
            uint2 code[kGatherRows][2];
            uint32_t sc[kGatherRows][2];
            #pragma unroll
            for (int r = 0; r < kGatherRows; ++r) {
                #pragma unroll
                for (int h = 0; h < 2; ++h) {
                    code[r][h] = make_uint2(0u, 0u);
                    sc[r][h] = 127;
                    if (at[r] >= 0) {
                        const uint8_t *p = pool.base + at[r];
                        code[r][h] = *reinterpret_cast<const uint2 *>(
                            p + (int64_t)o[r] * kLatent + 256 * h + 8 * lane);
                        sc[r][h] = p[(int64_t)pool.page_size * (kLatent + 2 * kLatRope) +
                                     (int64_t)o[r] * kLatGroups + 4 * h + (lane >> 3)];
                    }
                }
            }
            // the rotated elements: eight lanes a row
            uint4 rope = make_uint4(0u, 0u, 0u, 0u);
            const int64_t ra = __shfl_sync(0xffffffffu, place, lane >> 3);
            const int ro = __shfl_sync(0xffffffffu, off, lane >> 3);
            if (ra >= 0)
                rope = *reinterpret_cast<const uint4 *>(
                    pool.base + ra + (int64_t)pool.page_size * kLatent +
                    (int64_t)ro * 2 * kLatRope + 16 * (lane & 7));
            #pragma unroll
            for (int r = 0; r < kGatherRows; ++r) {
                if (r >= live)
                    break;
                #pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float s = e8m0_float(sc[r][h]);
                    const uint2 a = codes_to_bf16(code[r][h].x, s);
                    const uint2 b = codes_to_bf16(code[r][h].y, s);
                    *reinterpret_cast<uint4 *>(out + (first + r) * ld_out + 256 * h + 8 * lane) =
                        make_uint4(a.x, a.y, b.x, b.y);
                }
            }
            if ((lane >> 3) < live)
                *reinterpret_cast<uint4 *>(out + (first + (lane >> 3)) * ld_out + kLatent +
                                           8 * (lane & 7)) = rope;
        } else {
            // 72 pieces of 16 bytes a row
            constexpr int kPieces = kLatBf16TokBytes / 16;
            uint4 v[kGatherRows][3];
            #pragma unroll
            for (int r = 0; r < kGatherRows; ++r) {
                #pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const int p = 32 * i + lane;
                    v[r][i] = make_uint4(0u, 0u, 0u, 0u);
                    if (at[r] >= 0 && p < kPieces)
                        v[r][i] = *reinterpret_cast<const uint4 *>(
                            pool.base + at[r] + (int64_t)o[r] * kLatBf16TokBytes + 16 * p);
                }
            }
            #pragma unroll
            for (int r = 0; r < kGatherRows; ++r) {
                if (r >= live)
                    break;
                #pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const int p = 32 * i + lane;
                    if (p < kPieces)
                        *reinterpret_cast<uint4 *>(out + (first + r) * ld_out + 8 * p) = v[r][i];
                }
            }
        }
    }
}

// One warp per `per_warp` tokens, at most 16 CTAs per SM (a full SM of warps).
int cache_grid(long long tokens, int per_warp)
{
    const long long ctas = (tokens + (kCacheThreads / 32) * per_warp - 1) /
                           ((kCacheThreads / 32) * per_warp);
    const long long cap = (long long)sm_count() * 16;
    return (int)(ctas < cap ? ctas : cap);
}

} // namespace
} // namespace idx

using namespace idx;

extern "C" idx_status idx_latent_store(const uint16_t *kv, int64_t ld_kv, const int32_t *positions,
                                       const float *cos_sin, int64_t ld_cos_sin,
                                       int num_positions, const float *norm_weight, float eps,
                                       int T, int L, int rope_dim, idx_latent_format fmt,
                                       uint8_t *kv_pages, int64_t page_stride_bytes,
                                       int num_pages, int page_size, const int64_t *slot_mapping,
                                       idx_stream_t stream)
{
    IDX_NVTX_RANGE("idx_latent_store");
    if (T < 0 || L <= 0 || rope_dim < 0 || ld_kv < (int64_t)L + rope_dim || !(eps >= 0.0f) ||
        (cos_sin && (num_positions < 0 || ld_cos_sin < rope_dim)))
        return IDX_ERR_INVALID_ARG;
    if (T == 0)
        return IDX_OK;
    if (!kv || !slot_mapping || (cos_sin && !positions))
        return IDX_ERR_INVALID_ARG;
    if (L != kLatent || rope_dim != kLatRope)
        return IDX_ERR_UNSUPPORTED;
    const idx_status ok = check_pool(kv_pages, page_stride_bytes, num_pages, page_size, fmt);
    if (ok != IDX_OK)
        return ok;
    if (!aligned16(kv) || ld_kv % 8 != 0 || (norm_weight && !aligned16(norm_weight)))
        return IDX_ERR_UNSUPPORTED;
    unsigned int *status = device_status_ptr();
    if (!status)
        return IDX_ERR_CUDA;
    auto kern = fmt == IDX_LATENT_FP8_E4M3 ? latent_store_kernel<true> : latent_store_kernel<false>;
    return launch_status(launch_pdl(
        kern, dim3(cache_grid(T, 1)), dim3(kCacheThreads), 0, (cudaStream_t)stream, kv, ld_kv,
        positions, cos_sin, ld_cos_sin, num_positions, norm_weight, eps, T,
        make_pool(kv_pages, page_stride_bytes, num_pages, page_size), slot_mapping, status));
}

extern "C" idx_status idx_latent_gather(const uint8_t *kv_pages, int64_t page_stride_bytes,
                                        int num_pages, int page_size, idx_latent_format fmt,
                                        int L, int rope_dim, const int32_t *block_table,
                                        int64_t bt_stride, int max_blocks,
                                        const int32_t *cu_lens, const int32_t *seq_starts, int B,
                                        int N, uint16_t *out, int64_t ld_out, idx_stream_t stream)
{
    IDX_NVTX_RANGE("idx_latent_gather");
    if (L <= 0 || rope_dim < 0 || B < 0 || N < 0 || max_blocks < 0 || bt_stride < max_blocks ||
        ld_out < (int64_t)L + rope_dim)
        return IDX_ERR_INVALID_ARG;
    if (N == 0 || B == 0)
        return IDX_OK;
    if (!block_table || !cu_lens || !out)
        return IDX_ERR_INVALID_ARG;
    if (L != kLatent || rope_dim != kLatRope)
        return IDX_ERR_UNSUPPORTED;
    const idx_status ok = check_pool(kv_pages, page_stride_bytes, num_pages, page_size, fmt);
    if (ok != IDX_OK)
        return ok;
    if (!aligned16(out) || ld_out % 8 != 0)
        return IDX_ERR_UNSUPPORTED;
    unsigned int *status = device_status_ptr();
    if (!status)
        return IDX_ERR_CUDA;
    auto kern =
        fmt == IDX_LATENT_FP8_E4M3 ? latent_gather_kernel<true> : latent_gather_kernel<false>;
    return launch_status(launch_pdl(
        kern, dim3(cache_grid(N, kGatherRows)), dim3(kCacheThreads), 0, (cudaStream_t)stream,
        make_pool(kv_pages, page_stride_bytes, num_pages, page_size), block_table, bt_stride,
        max_blocks, cu_lens, seq_starts, B, N, out, ld_out, status));
}
