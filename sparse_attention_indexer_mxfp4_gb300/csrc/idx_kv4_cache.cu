// idx_kv4_cache.cu -- the 4-bit cache's writer, its read-back and the eviction
// that moves the tokens that stay to other pages.
#include <algorithm>
#include <atomic>
#include <climits>

#include "idx_kv4.cuh"
#include "idx_topk_cluster.cuh"

namespace idx {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
// Items (a token's keys and values of one head) whose loads a warp has in flight
// (8191 tokens x 8 heads written and read back: four 21.2 us, eight 27.1, two 25.7);
// where there are fewer than fill the SMs, one (128 tokens 5.0 -> 4.3 us).
constexpr int kItemsMany = 4;
constexpr int kShortSum = 2048;  // columns of a summed list that one CTA selects from

// ----------------------------------------------------------------- the store
//
// A half warp a token's keys of one head, the other its values, eight elements
// a lane; a group's four lanes share its largest magnitude.  The exponent is
// the least with amax / 2^e <= 6 = 1.5 * 2^2, read off the bits: one more
// where the mantissa is over 1.5.  Scaling by a power of two is exact, so the
// hardware's conversion (nearest, ties to even) rounds the element itself.
// Bound: 512 bytes in, 136 out a token and head.

__device__ __forceinline__ uint32_t quantise8(uint4 raw, int &bits)
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t top = 0x00800000u;  // 2^-126
    #pragma unroll
    for (int i = 0; i < 4; ++i)  // as integers, so that a NaN counts as the largest
        top = max(top, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (top >= 0x7f800000u) {
        bits = 255;
        return 0;
    }
    bits = max(0, (int)(top >> 23) - 2 + ((top & 0x7fffffu) > 0x400000u));
    // 2^(127 - bits) (the largest finite magnitude has 253)
    const float inv = __uint_as_float((uint32_t)(254 - bits) << 23);
    uint32_t out = 0;
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(w[i] << 16) * inv,
                    b = __uint_as_float(w[i] & 0xffff0000u) * inv;
        uint32_t two;  // the second source lands in the low nibble
        asm("{\n\t.reg .b8 c;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\t"
            "mov.b32 %0, {c, 0, 0, 0};\n\t}"
            : "=r"(two)
            : "f"(a), "f"(b));
        out |= two << (8 * i);
    }
    return out;
}

struct Kv4Rows {
    const uint16_t *k, *v;
    int64_t ldk_row, ldk_head, ldv_row, ldv_head;
};

template <int kItems>
__global__ void __launch_bounds__(kThreads)
    kv4_store_kernel(const Kv4Rows in, uint32_t items, const Kv4Pool pool,
                     const int64_t *__restrict__ slots, unsigned int *status)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = lane_id(), side = lane >> 4, piece = lane & 15;
    const uint16_t *src = side ? in.v : in.k;
    const int64_t ld_row = side ? in.ldv_row : in.ldk_row;
    const int64_t ld_head = side ? in.ldv_head : in.ldk_head;
    const uint32_t step = gridDim.x * kWarps * kItems;
    for (uint32_t i0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kItems; i0 < items; i0 += step) {
        uint4 raw[kItems];
        int64_t slot[kItems];
        int head[kItems];
        #pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const uint32_t it = i0 + i, t = it / (uint32_t)pool.heads;
            const int h = head[i] = (int)(it - t * pool.heads);
            slot[i] = -1;
            raw[i] = make_uint4(0u, 0u, 0u, 0u);
            if (it < items) {
                slot[i] = slots[t];
                raw[i] = *reinterpret_cast<const uint4 *>(src + t * ld_row + h * ld_head + 8 * piece);
            }
        }
        #pragma unroll
        for (int i = 0; i < kItems; ++i) {
            int bits;
            const uint32_t codes = quantise8(raw[i], bits);
            if (slot[i] < 0)
                continue;
            if (slot[i] >= (int64_t)pool.p.num_pages * pool.p.page_size) {
                if (lane == 0)
                    atomicOr(status, kDevBadPage);
                continue;
            }
            const int page = page_of(pool.p, (int)slot[i]);
            const int off = (int)slot[i] - page * pool.p.page_size;
            const int h = head[i];
            uint8_t *base = const_cast<uint8_t *>(pool.p.base);
            *reinterpret_cast<uint32_t *>(base + kv4_codes_at(pool, page, h, off) +
                                          side * pool.side + 4 * piece) = codes;
            if ((lane & 3) == 0)
                base[kv4_scales_at(pool, page, h, off) + side * pool.scale_side + (piece >> 2)] =
                    (uint8_t)bits;
        }
    }
}

// ------------------------------------------------------------- the read-back
//
// The same shape the other way: a lane a word of codes, sixteen bytes of bf16
// out.  A code times a power of two has two significant bits, so bf16 holds it
// exactly.

template <int kItems>
__global__ void __launch_bounds__(kThreads)
    kv4_gather_kernel(const Kv4Pool pool, const int32_t *__restrict__ table, int64_t bt_stride,
                      int max_blocks, const int32_t *__restrict__ cu,
                      const int32_t *__restrict__ starts, int B, int N, uint16_t *k_out,
                      int64_t ldk_row, int64_t ldk_head, uint16_t *v_out, int64_t ldv_row,
                      int64_t ldv_head, unsigned int *status)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = lane_id(), side = lane >> 4, piece = lane & 15;
    uint16_t *dst = side ? v_out : k_out;
    const int64_t ld_row = side ? ldv_row : ldk_row, ld_head = side ? ldv_head : ldk_head;
    const int end = cu[B];
    if (blockIdx.x == 0 && threadIdx.x == 0 && (end < 0 || end > N))
        atomicOr(status, kDevBadBounds);
    // (products with parts are unsigned: a bound below zero would wrap)
    const uint32_t rows = max(0, min(N, end));
    // a warp has the heads of a row, kItems at a time
    const uint32_t parts = (pool.heads + kItems - 1) / kItems;
    const uint32_t step = gridDim.x * kWarps;
    for (uint32_t i = blockIdx.x * kWarps + (threadIdx.x >> 5); i < rows * parts; i += step) {
        const int n = (int)(i / parts), h0 = (int)(i - n * parts) * kItems;
        int lo = 0, hi = B - 1;  // the first sequence that ends past row n
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid + 1] > n)
                hi = mid;
            else
                lo = mid + 1;
        }
        const int64_t t = (int64_t)n - cu[lo] + (starts ? starts[lo] : 0);
        int page = -1, off = 0;
        if (t >= 0 && t < (int64_t)max_blocks * pool.p.page_size && t <= INT_MAX) {
            const int block = page_of(pool.p, (int)t);
            off = (int)t - block * pool.p.page_size;
            page = table[lo * bt_stride + block];
            if (page < 0 || page >= pool.p.num_pages)
                page = -1;
        }
        if (page < 0 && lane == 0)
            atomicOr(status, kDevBadPage);
        uint32_t code[kItems];
        uint8_t bits[kItems];
        #pragma unroll
        for (int k = 0; k < kItems; ++k) {
            code[k] = 0;
            bits[k] = 0;
            if (page >= 0 && h0 + k < pool.heads) {
                code[k] = *reinterpret_cast<const uint32_t *>(
                    pool.p.base + kv4_codes_at(pool, page, h0 + k, off) + side * pool.side + 4 * piece);
                bits[k] = pool.p.base[kv4_scales_at(pool, page, h0 + k, off) +
                                      side * pool.scale_side + (piece >> 2)];
            }
        }
        #pragma unroll
        for (int k = 0; k < kItems; ++k) {
            if (h0 + k >= pool.heads)
                break;
            float s[4];
            e8m0_to_float(bits[k], s);
            uint32_t h[4], o[4];
            e2m1_to_f16x2(code[k], h);
            #pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
                const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s[0], f.y * s[0]);
                o[e] = *reinterpret_cast<const uint32_t *>(&b);
            }
            *reinterpret_cast<uint4 *>(dst + n * ld_row + (h0 + k) * ld_head + 8 * piece) =
                make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// -------------------------------------------------------------- the eviction
//
// A cluster of CTAs a list selects among the tokens that are not recent: the
// cluster form of the top-k on weights, of a head or summed over the heads, which
// stay in its shared memory.  Then the tokens that stay go to their new places.
// Tokens move to pages of their own: the old ones may belong to other sequences
// too.  Bound: the weights once, the tokens that stay read and written (136 bytes).
//
// A sum over heads is of pairs of floats (sum and what it lost to rounding, 48 bits
// together), rounded once; 64-bit additions are so few a clock that they bounded the
// selection (32 contexts x 8 heads 31 us).  Longer contexts than a cluster holds
// take scores in scratch and the general top-k.

struct EvictArgs {
    const float *mass;
    int64_t ld_batch, ld_head;
    int ld;  // columns
    const int32_t *ctx;
    int B, heads, lists;  // lists: of a sequence, its heads or one
    int budget, recent;
    float *score;
    int64_t ld_score;
    int32_t *lengths;
    int32_t *keep;  // [B, lists, budget]
    int32_t *new_ctx;
    float *new_mass;  // [B, heads, budget]
    const int32_t *table, *new_table;
    int64_t bt_stride, new_stride;
    int blocks, new_blocks;
    unsigned int *status;
};

// Tokens of a sequence; the weights' columns bound it.
__device__ __forceinline__ int evict_len(const EvictArgs &a, int b)
{
    return min(max(a.ctx[b], 0), a.ld);
}

// What the top-k orders by: finite numbers (it passes over others), infinities as the
// largest and the least of them, NaN as the least, zeros of either sign as one.
__device__ __forceinline__ float orderly(float x)
{
    constexpr float most = 3.402823466e38f;
    return x != x ? -most : fminf(fmaxf(x, -most), most) + 0.0f;
}

// a + b as a float and what the float lacks.
__device__ __forceinline__ void add_pair(float &hi, float &lo, float b)
{
    const float sum = hi + b, part = sum - hi;
    lo += (hi - (sum - part)) + (b - part);
    hi = sum;
}

__device__ __forceinline__ float of_pair(float hi, float lo)
{
    return isfinite(hi) ? hi + lo : hi;  // (infinities leave NaN behind)
}

// Weight of token t of a list.
__device__ __forceinline__ float evict_weight(const EvictArgs &a, const float *m, int t)
{
    if (a.lists == a.heads)
        return m[t];
    float hi = 0.0f, lo = 0.0f;
    #pragma unroll 8
    for (int h = 0; h < a.heads; ++h)
        add_pair(hi, lo, m[h * a.ld_head + t]);
    return of_pair(hi, lo);
}

// The keys of a list for the top-k's cluster form.
struct Weights {
    static constexpr bool kRuns = true;
    EvictArgs a;
    int vec_ok;  // four columns side by side are one load

    __device__ __forceinline__ int len(int row) const
    {
        const int n = evict_len(a, row / a.lists);
        return n > a.budget ? n - a.recent : 0;
    }
    __device__ __forceinline__ void run(int row, int base, int at, int end, uint32_t (&key)[4]) const
    {
        const int b = row / a.lists, g = row - b * a.lists;
        const float *m = a.mass + b * a.ld_batch + g * a.ld_head + base;
        float x[4] = {};
        if (vec_ok && at + 4 <= end) {
            const int heads = a.lists == a.heads ? 1 : a.heads;
            float lo[4] = {};
            for (int h0 = 0; h0 < heads; h0 += 4) {
                float4 v[4];
                #pragma unroll
                for (int h = 0; h < 4; ++h)
                    v[h] = h0 + h < heads
                               ? __ldg(reinterpret_cast<const float4 *>(m + (h0 + h) * a.ld_head + at))
                               : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                #pragma unroll
                for (int h = 0; h < 4; ++h) {
                    add_pair(x[0], lo[0], v[h].x);
                    add_pair(x[1], lo[1], v[h].y);
                    add_pair(x[2], lo[2], v[h].z);
                    add_pair(x[3], lo[3], v[h].w);
                }
            }
            #pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = of_pair(x[e], lo[e]);
        } else {
            #pragma unroll
            for (int e = 0; e < 4; ++e)
                if (at + e < end)
                    x[e] = evict_weight(a, m, at + e);
        }
        #pragma unroll
        for (int e = 0; e < 4; ++e)
            key[e] = at + e < end ? order_key(orderly(x[e])) : 0u;
    }
};

// Short lists, of single heads or (kSum) summed over them: a CTA each, the keys in
// its registers (4 sequences x 8 heads of up to 8192 tokens to 2048 in clusters 16.9
// us, here 10.4).
template <bool kSum>
__global__ void __launch_bounds__(topk_short::kThreads, 3)
    evict_short_kernel(const Weights src, int k, int32_t *__restrict__ out, int64_t ld_out)
{
    namespace T = topk_short;
    __shared__ __align__(16) regsel::Shared<T::kThreads, T::kSteps> sh;
    const int row = blockIdx.x, tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    const int len = src.len(row), nrun = (len + 4 * T::kThreads - 1) / (4 * T::kThreads);
    const EvictArgs &a = src.a;
    uint32_t key[T::kSteps][4];
    if constexpr (kSum) {
        #pragma unroll
        for (int s = 0; s < T::kSteps; ++s) {
            key[s][0] = key[s][1] = key[s][2] = key[s][3] = 0u;
            if (s < nrun)
                src.run(row, 0, 4 * (s * T::kThreads + tid), len, key[s]);
        }
        regsel::select_write<T::kThreads, T::kSteps>(
            sh, key, k, out + (size_t)row * ld_out,
            [&](int s, int e) -> int32_t { return s * 4 * T::kThreads + 4 * tid + e; }, nrun);
        return;
    }
    const float *m = a.mass + row / a.heads * a.ld_batch + row % a.heads * a.ld_head;
    float4 v[T::kSteps];
    #pragma unroll
    for (int s = 0; s < T::kSteps; ++s) {
        const int at = 4 * (s * T::kThreads + tid);
        v[s] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (src.vec_ok && at + 4 <= len) {
            v[s] = __ldg(reinterpret_cast<const float4 *>(m + at));
        } else {
            v[s].x = at < len ? __ldg(m + at) : 0.0f;
            v[s].y = at + 1 < len ? __ldg(m + at + 1) : 0.0f;
            v[s].z = at + 2 < len ? __ldg(m + at + 2) : 0.0f;
            v[s].w = at + 3 < len ? __ldg(m + at + 3) : 0.0f;
        }
    }
    #pragma unroll
    for (int s = 0; s < T::kSteps; ++s) {
        const int at = 4 * (s * T::kThreads + tid);
        const float x[4] = {v[s].x, v[s].y, v[s].z, v[s].w};
        #pragma unroll
        for (int e = 0; e < 4; ++e)
            key[s][e] = at + e < len ? order_key(orderly(x[e])) : 0u;
    }
    regsel::select_write<T::kThreads, T::kSteps>(
        sh, key, k, out + (size_t)row * ld_out,
        [&](int s, int e) -> int32_t { return s * 4 * T::kThreads + 4 * tid + e; }, nrun);
}

// The same in scratch.
__global__ void __launch_bounds__(kThreads) evict_score_kernel(const EvictArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const int row = blockIdx.y, b = row / a.lists, g = row - b * a.lists;
    const int n = evict_len(a, b), old = n > a.budget ? n - a.recent : 0;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        a.lengths[row] = old;
    const float *m = a.mass + b * a.ld_batch + g * a.ld_head;
    for (int t = blockIdx.x * kThreads + threadIdx.x; t < old; t += gridDim.x * kThreads)
        a.score[row * a.ld_score + t] = orderly(evict_weight(a, m, t));
}

// 32 tokens of a head a warp: a lane looks a token up, four lanes move its 64
// bytes of keys, then of values (eight tokens at once, all loads before the first
// store: 4 KB in flight a warp), a lane each its scales and weight.  A warp each: CTAs
// that walk on instead took 136 us where these take 130, with the next tokens looked
// up ahead 142 (32 contexts x 8 heads to 8192 tokens, selection and all).
__global__ void __launch_bounds__(kThreads) evict_move_kernel(const EvictArgs a, const Kv4Pool pool)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = lane_id();
    const uint32_t parts = max(1, (a.budget + 31) / 32);
    uint8_t *base = const_cast<uint8_t *>(pool.p.base);
    const uint32_t i = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (i < a.B * a.heads * parts) {
        const int bh = (int)(i / parts), j0 = (int)(i - bh * parts) * 32;
        const int b = bh / a.heads, h = bh - b * a.heads, g = a.lists == 1 ? 0 : h;
        const int n = evict_len(a, b), kept = min(n, a.budget), chosen = a.budget - a.recent;
        if (h == 0 && j0 == 0 && lane == 0) {
            a.new_ctx[b] = kept;
            if (a.ctx[b] < 0 || a.ctx[b] > a.ld)
                atomicOr(a.status, kDevBadBounds);
        }
        // this lane's token: its place and its new one
        const int j = j0 + lane;
        int32_t *list = a.keep + ((int64_t)b * a.lists + g) * a.budget;
        const bool listed = n > a.budget && j < chosen;  // by the top-k
        int src = -1;
        if (j < kept)
            src = n <= a.budget ? j : listed ? list[j] : n - a.recent + (j - chosen);
        if (j < a.budget && !listed && h == g)
            list[j] = src;
        int64_t from = -1, to = -1, sc_from = 0, sc_to = 0;
        float m = 0.0f;
        if (src >= 0) {
            const int sb = page_of(pool.p, src), db = page_of(pool.p, j);
            const int sp = sb < a.blocks ? a.table[b * a.bt_stride + sb] : -1;
            const int dp = db < a.new_blocks ? a.new_table[b * a.new_stride + db] : -1;
            m = a.mass[b * a.ld_batch + h * a.ld_head + src];
            if (sp >= 0 && sp < pool.p.num_pages) {
                from = kv4_codes_at(pool, sp, h, src - sb * pool.p.page_size);
                sc_from = kv4_scales_at(pool, sp, h, src - sb * pool.p.page_size);
            }
            if (dp >= 0 && dp < pool.p.num_pages) {
                to = kv4_codes_at(pool, dp, h, j - db * pool.p.page_size);
                sc_to = kv4_scales_at(pool, dp, h, j - db * pool.p.page_size);
            }
            if (from < 0 || to < 0)
                atomicOr(a.status, kDevBadPage);
        }
        uint4 kv[4][2] = {};
        uint32_t sc[2] = {};
        #pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int64_t at = __shfl_sync(0xffffffffu, from, 8 * x + (lane >> 2));
            if (at >= 0) {
                kv[x][0] = *reinterpret_cast<const uint4 *>(base + at + 16 * (lane & 3));
                kv[x][1] = *reinterpret_cast<const uint4 *>(base + at + pool.side + 16 * (lane & 3));
            }
        }
        if (from >= 0) {
            sc[0] = *reinterpret_cast<const uint32_t *>(base + sc_from);
            sc[1] = *reinterpret_cast<const uint32_t *>(base + sc_from + pool.scale_side);
        }
        #pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int64_t at = __shfl_sync(0xffffffffu, to, 8 * x + (lane >> 2));
            if (at >= 0) {
                *reinterpret_cast<uint4 *>(base + at + 16 * (lane & 3)) = kv[x][0];
                *reinterpret_cast<uint4 *>(base + at + pool.side + 16 * (lane & 3)) = kv[x][1];
            }
        }
        if (to >= 0) {
            *reinterpret_cast<uint32_t *>(base + sc_to) = sc[0];
            *reinterpret_cast<uint32_t *>(base + sc_to + pool.scale_side) = sc[1];
        }
        if (j < a.budget)
            a.new_mass[(int64_t)bh * a.budget + j] = m;
    }
}

// Selection without scratch.  The cluster form has as many CTAs a list as there are
// SMs for, and at least enough to hold it; none with less than half a run of keys
// (2048).
cudaError_t select_on_chip(const EvictArgs &a, int chosen, cudaStream_t stream)
{
    namespace T = topk_cluster;
    const int rows = a.B * a.lists;
    const int vec_ok = (a.ld_batch | a.ld_head) % 4 == 0 && aligned16(a.mass);
    if (a.lists == a.heads && a.ld <= topk_short::kMaxLen)
        return launch_pdl(evict_short_kernel<false>, dim3(rows), dim3(topk_short::kThreads), 0, stream,
                          Weights{a, vec_ok}, chosen, a.keep, (int64_t)a.budget);
    // (a CTA alone reads a run of a few heads' weights in about a microsecond)
    if (a.ld <= kShortSum)
        return launch_pdl(evict_short_kernel<true>, dim3(rows), dim3(topk_short::kThreads), 0, stream,
                          Weights{a, vec_ok}, chosen, a.keep, (int64_t)a.budget);
    const int least = (a.ld + T::kChunk - 1) / T::kChunk, most = (a.ld + 2047) / 2048;
    const int C = std::max(least, std::min({T::kMaxCluster, most, sm_count() / rows}));
    static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(T::topk_cluster_kernel<Weights>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(T::Shared));
        if (e != cudaSuccess)
            return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(T::kThreads);
    cfg.dynamicSmemBytes = sizeof(T::Shared);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, T::topk_cluster_kernel<Weights>, Weights{a, vec_ok}, rows, chosen,
                              a.keep, (int64_t)a.budget, SlotCount{});
}

// CTAs for so many warps of work, at most a full SM of warps each.
int grid_of(int64_t warps)
{
    return (int)std::min<int64_t>((warps + kWarps - 1) / kWarps, (int64_t)sm_count() * 8);
}

// Items a warp for so many of them.
int items_of(int64_t items)
{
    return items > (int64_t)sm_count() * 4 * kWarps ? kItemsMany : 1;
}

// Where the parts of the eviction's scratch begin.
struct EvictScratch {
    int64_t ld_score;
    size_t lengths, topk, all;

    EvictScratch(int B, int lists, int ld, int chosen)
    {
        const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
        const size_t rows = (size_t)B * lists;
        ld_score = ((int64_t)ld + 3) / 4 * 4;
        lengths = up(rows * ld_score * sizeof(float));
        topk = lengths + up(rows * sizeof(int32_t));
        all = topk + up(chosen > 0 && rows <= INT_MAX
                            ? idx_topk_workspace_size((int)rows, ld_score, chosen) : 0);
    }
};

} // namespace
} // namespace idx

using namespace idx;

extern "C" idx_status idx_kv4_store(const uint16_t *k, int64_t ldk_row, int64_t ldk_head,
                                    const uint16_t *v, int64_t ldv_row, int64_t ldv_head, int T,
                                    int kv_heads, int D, uint8_t *kv_pages,
                                    int64_t page_stride_bytes, int num_pages, int page_size,
                                    const int64_t *slot_mapping, idx_stream_t stream)
{
    IDX_NVTX_RANGE("idx_kv4_store");
    if (T < 0 || kv_heads <= 0 || D <= 0 || ldk_head < D || ldk_row < 0 || ldv_head < D ||
        ldv_row < 0)
        return IDX_ERR_INVALID_ARG;
    if (T == 0)
        return IDX_OK;
    if (!k || !v || !slot_mapping)
        return IDX_ERR_INVALID_ARG;
    if (D != kKv4Dim)
        return IDX_ERR_UNSUPPORTED;
    const idx_status ok = check_kv4_pool(kv_pages, page_stride_bytes, num_pages, page_size, kv_heads);
    if (ok != IDX_OK)
        return ok;
    const int64_t items = (int64_t)T * kv_heads;
    if (!aligned16(k) || !aligned16(v) || (ldk_row | ldk_head | ldv_row | ldv_head) % 8 != 0 ||
        items > INT32_MAX)
        return IDX_ERR_UNSUPPORTED;
    unsigned int *status = device_status_ptr();
    if (!status)
        return IDX_ERR_CUDA;
    const int each = items_of(items);
    return launch_status(launch_pdl(
        each == 1 ? kv4_store_kernel<1> : kv4_store_kernel<kItemsMany>,
        dim3(grid_of((items + each - 1) / each)), dim3(kThreads), 0,
        (cudaStream_t)stream, Kv4Rows{k, v, ldk_row, ldk_head, ldv_row, ldv_head}, (uint32_t)items,
        make_kv4_pool(kv_pages, page_stride_bytes, num_pages, page_size, kv_heads), slot_mapping,
        status));
}

extern "C" idx_status idx_kv4_gather(const uint8_t *kv_pages, int64_t page_stride_bytes,
                                     int num_pages, int page_size, int kv_heads, int D,
                                     const int32_t *block_table, int64_t bt_stride, int max_blocks,
                                     const int32_t *cu_lens, const int32_t *seq_starts, int B,
                                     int N, uint16_t *k_out, int64_t ldk_row, int64_t ldk_head,
                                     uint16_t *v_out, int64_t ldv_row, int64_t ldv_head,
                                     idx_stream_t stream)
{
    IDX_NVTX_RANGE("idx_kv4_gather");
    if (kv_heads <= 0 || D <= 0 || B < 0 || N < 0 || max_blocks < 0 || bt_stride < max_blocks ||
        ldk_head < D || ldk_row < 0 || ldv_head < D || ldv_row < 0)
        return IDX_ERR_INVALID_ARG;
    if (N == 0 || B == 0)
        return IDX_OK;
    if (!block_table || !cu_lens || !k_out || !v_out)
        return IDX_ERR_INVALID_ARG;
    if (D != kKv4Dim)
        return IDX_ERR_UNSUPPORTED;
    const idx_status ok = check_kv4_pool(kv_pages, page_stride_bytes, num_pages, page_size, kv_heads);
    if (ok != IDX_OK)
        return ok;
    if (!aligned16(k_out) || !aligned16(v_out) ||
        (ldk_row | ldk_head | ldv_row | ldv_head) % 8 != 0 || (int64_t)N * kv_heads > INT32_MAX)
        return IDX_ERR_UNSUPPORTED;
    const Strided keys = {k_out, N, ldk_row, kv_heads, ldk_head, D, 2};
    const Strided values = {v_out, N, ldv_row, kv_heads, ldv_head, D, 2};
    if (!lie_apart(keys) || !lie_apart(values) || !lie_apart(keys, values))
        return IDX_ERR_INVALID_ARG;
    unsigned int *status = device_status_ptr();
    if (!status)
        return IDX_ERR_CUDA;
    const int each = items_of((int64_t)N * kv_heads);
    return launch_status(launch_pdl(
        each == 1 ? kv4_gather_kernel<1> : kv4_gather_kernel<kItemsMany>,
        dim3(grid_of((int64_t)N * ((kv_heads + each - 1) / each))), dim3(kThreads), 0, (cudaStream_t)stream,
        make_kv4_pool(kv_pages, page_stride_bytes, num_pages, page_size, kv_heads), block_table,
        bt_stride, max_blocks, cu_lens, seq_starts, B, N, k_out, ldk_row, ldk_head, v_out, ldv_row,
        ldv_head, status));
}

extern "C" size_t idx_kv4_evict_workspace_size(int B, int kv_heads, int ld_mass, int budget,
                                               int recent, int whole_tokens)
{
    // nothing is chosen, or a cluster holds what it is chosen from
    if (B <= 0 || kv_heads <= 0 || ld_mass <= budget || budget <= recent ||
        ld_mass <= topk_cluster::kMaxLen)
        return 0;
    return EvictScratch(B, whole_tokens ? 1 : kv_heads, ld_mass, budget - recent).all;
}

extern "C" int idx_kv4_evict_launches(int B, int kv_heads, int ld_mass, int budget, int recent,
                                      int whole_tokens)
{
    if (B <= 0 || kv_heads <= 0)
        return 0;
    if (ld_mass <= budget || budget <= recent)
        return 1;
    if (ld_mass <= topk_cluster::kMaxLen)
        return 2;
    const int lists = whole_tokens ? 1 : kv_heads;
    const EvictScratch at(B, lists, ld_mass, budget - recent);
    return at.all > at.topk ? 4 : 3;  // the top-k with scratch of its own is two kernels
}

extern "C" idx_status idx_kv4_evict(const float *mass, int64_t ld_batch, int64_t ld_head,
                                    int ld_mass, const int32_t *context_lens, int B, int kv_heads,
                                    int D, int budget, int recent, int whole_tokens,
                                    uint8_t *kv_pages, int64_t page_stride_bytes, int num_pages,
                                    int page_size, const int32_t *block_table, int64_t bt_stride,
                                    int max_blocks, const int32_t *new_table, int64_t new_stride,
                                    int new_blocks, int32_t *keep, int32_t *new_lens,
                                    float *new_mass, void *ws, size_t ws_bytes, idx_stream_t stream)
{
    IDX_NVTX_RANGE("idx_kv4_evict");
    if (B < 0 || kv_heads <= 0 || D <= 0 || ld_mass < 0 || budget < 0 || recent < 0 ||
        recent > budget || ld_head < 0 || ld_batch < 0 || max_blocks < 0 || bt_stride < max_blocks ||
        new_blocks < 0 || new_stride < new_blocks)
        return IDX_ERR_INVALID_ARG;
    if (B == 0)
        return IDX_OK;
    if ((!mass && ld_mass > 0) || !context_lens || !new_lens ||
        (budget > 0 && (!block_table || !new_table || !keep || !new_mass)))
        return IDX_ERR_INVALID_ARG;
    if (D != kKv4Dim)
        return IDX_ERR_UNSUPPORTED;
    const idx_status ok = check_kv4_pool(kv_pages, page_stride_bytes, num_pages, page_size, kv_heads);
    if (ok != IDX_OK)
        return ok;
    if ((int64_t)new_blocks * page_size < std::min(budget, ld_mass))
        return IDX_ERR_INVALID_ARG;  // no room for what stays
    const int lists = whole_tokens ? 1 : kv_heads;
    // rows are a grid's second dimension
    if ((int64_t)B * lists > 65535 || ld_mass > INT32_MAX - 3 ||
        (int64_t)B * kv_heads > INT32_MAX / ((int64_t)budget + 32))
        return IDX_ERR_UNSUPPORTED;
    const size_t need =
        idx_kv4_evict_workspace_size(B, kv_heads, ld_mass, budget, recent, whole_tokens);
    if (need > 0 && (!ws || !aligned16(ws) || ws_bytes < need))
        return IDX_ERR_WORKSPACE;
    // every part of the call reads the inputs while others write: no output may be one of them
    struct Bytes {
        const void *p;
        __int128 n;
    };
    const Bytes parts[] = {
        {keep, (__int128)4 * B * lists * budget},
        {new_lens, (__int128)4 * B},
        {new_mass, (__int128)4 * B * kv_heads * budget},
        {mass, span({mass, B, ld_batch, kv_heads, ld_head, ld_mass, 4})},
        {context_lens, (__int128)4 * B},
        {block_table, span({block_table, B, bt_stride, 1, 0, max_blocks, 4})},
        {new_table, span({new_table, B, new_stride, 1, 0, new_blocks, 4})}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 7; ++j)
            if (meet(parts[i].p, parts[i].n, parts[j].p, parts[j].n))
                return IDX_ERR_INVALID_ARG;
    EvictArgs a = {};
    a.mass = mass;
    a.ld_batch = ld_batch;
    a.ld_head = ld_head;
    a.ld = ld_mass;
    a.ctx = context_lens;
    a.B = B;
    a.heads = kv_heads;
    a.lists = lists;
    a.budget = budget;
    a.recent = recent;
    a.keep = keep;
    a.new_ctx = new_lens;
    a.new_mass = new_mass;
    a.table = block_table;
    a.new_table = new_table;
    a.bt_stride = bt_stride;
    a.new_stride = new_stride;
    a.blocks = max_blocks;
    a.new_blocks = new_blocks;
    a.status = device_status_ptr();
    if (!a.status)
        return IDX_ERR_CUDA;
    const Kv4Pool pool = make_kv4_pool(kv_pages, page_stride_bytes, num_pages, page_size, kv_heads);
    const int chosen = budget - recent;
    if (need == 0 && chosen > 0 && ld_mass > budget) {
        const cudaError_t e = select_on_chip(a, chosen, (cudaStream_t)stream);
        if (e != cudaSuccess)
            return launch_status(e);
    } else if (need > 0) {
        const int rows = B * lists;
        const EvictScratch at(B, lists, ld_mass, chosen);
        uint8_t *w = static_cast<uint8_t *>(ws);
        a.score = reinterpret_cast<float *>(w);
        a.ld_score = at.ld_score;
        a.lengths = reinterpret_cast<int32_t *>(w + at.lengths);
        // a few waves of CTAs in all, at least four columns a thread
        const int across = std::min((ld_mass + 4 * kThreads - 1) / (4 * kThreads),
                                    std::max(1, sm_count() * 16 / rows));
        cudaError_t e = launch_pdl(evict_score_kernel, dim3(across, rows), dim3(kThreads), 0,
                                   (cudaStream_t)stream, a);
        if (e != cudaSuccess)
            return launch_status(e);
        const size_t top = at.all - at.topk;
        const idx_status st = idx_topk(a.score, a.ld_score, rows, a.lengths, chosen, keep, budget,
                                       top ? w + at.topk : nullptr, top, stream);
        if (st != IDX_OK)
            return st;
    }
    return launch_status(launch_pdl(
        evict_move_kernel,
        dim3((unsigned)(((int64_t)B * kv_heads * std::max(1, (budget + 31) / 32) + kWarps - 1) / kWarps)),
        dim3(kThreads), 0, (cudaStream_t)stream, a, pool));
}
