// idx_latent_attn.cu -- absorbed latent attention over ragged slots or whole
// paged contexts:  s = scale * q . token,  out = softmax(s) . token[:512].
//
// Every head of a row reads the same tokens, so a tile of 64 tokens is one
// 64 x 576 matrix in shared memory that serves both products:
//
//     S^T [64 tokens x heads]   = K [64 x 576] . Q^T          (36 MMAs, M = 64)
//     O^T [512 latents x heads] += K[:, :512]^T . P^T         (4 x 4 MMAs, M = 128)
//
// with the tokens (first product) and the latents (second) on the MMA's M and
// the heads on its N: 16, 32 or 64 of them a CTA, so few heads waste no tensor
// work, the running sums O^T stay in tensor memory for a row's whole length
// (4 N columns), and the tile is read in place both times, K-major by its
// token rows and M-major by its latent columns (the same 128-byte swizzled
// rows describe both).  More than 64 heads are two groups, each a unit of its
// own; the second reads the tokens from L2.
//
// Work is split over a flat list of (row, head group, tile): every CTA (one
// per SM) takes an equal contiguous share, whatever the rows' lengths.  Rows
// that lie in one share are finished there; the others leave unnormalised sums
// with their maximum in scratch and a second kernel joins them in share order.
//
// Warps: 0-3 softmax and epilogue; 4-11 bring tokens in (slot -> page ->
// global loads; 8-bit codes are widened to bf16 on the way, exactly, by two
// shifts and a multiplication with a power of two); 12 loads queries and
// issues the first product; 13 issues the second.  Two tile stages.
//
// Softmax: in powers of two; a thread holds two tokens of N / 4 heads.  The
// running maximum of a head only has to keep 2^x in range, so it is raised
// (with a rescaling of O^T) when a score exceeds it by more than 2^40, which
// after a row's first tile is rare; 32-bit sums lose nothing by it.
#include <algorithm>
#include <atomic>

#include "idx_latent.cuh"

namespace idx {
namespace {

constexpr int kTile = 64;                          // tokens of a tile
constexpr int kChunks = kLatTok / 64;              // 128-byte columns of a token row
constexpr int kChunkBytes = kTile * 128;           // one column of all 64 tokens
constexpr int kStageBytes = kChunks * kChunkBytes; // 73728
constexpr int kSoftWarps = 4, kLoadWarps = 8;
constexpr int kWarpS = kSoftWarps + kLoadWarps, kWarpPV = kWarpS + 1;
constexpr int kThreads = (kWarpPV + 1) * 32;
constexpr int kMaxHeads = 128;
constexpr float kLazy = 40.0f;  // a score may exceed its running maximum by 2^40
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

struct AttnArgs {
    LatentPool pool;
    const int32_t *slots, *indptr;  // ragged rows (indptr null: paged)
    int64_t num_slots;
    const int32_t *block_table, *context_lens;
    int64_t bt_stride;
    int ctx_per_row, next_n, max_len;
    int R, H, groups;
    float scale_log2;  // scale * log2(e)
    uint16_t *out;
    int64_t ldo_row, ldo_head;
    float *lse;
    int64_t ld_lse;
    void *ws_place;  // int4 a CTA: the row, group and tile its share begins at
    float *ws_part;  // two segments a CTA: O^T, then maxima, then sums
    unsigned int *status;
};

// Where a row's tokens are listed, and how many it has.
struct Row {
    int64_t first;
    int n;
};

__device__ __forceinline__ Row row_of(const AttnArgs &a, int r)
{
    if (a.indptr) {
        const int64_t lo = min((int64_t)max(a.indptr[r], 0), a.num_slots);
        const int64_t hi = min((int64_t)max(a.indptr[r + 1], 0), a.num_slots);
        return {lo, (int)max((int64_t)0, hi - lo)};
    }
    const int b = r / a.next_n, j = r - b * a.next_n;
    const int end = a.ctx_per_row ? a.context_lens[r] : a.context_lens[b] - a.next_n + j + 1;
    return {b * a.bt_stride, min(max(end, 0), a.max_len)};
}

// A row without tokens still takes one (empty) tile: it has outputs.
__device__ __forceinline__ int tiles_of(int n)
{
    return n > kTile ? (n + kTile - 1) / kTile : 1;
}

// The slot of token t of a row; -1 when its page is negative.
__device__ __forceinline__ int64_t slot_of(const AttnArgs &a, const Row &w, int t)
{
    if (a.indptr)
        return a.slots[w.first + t];
    const int p = page_of(a.pool, t);
    const int id = a.block_table[w.first + p];
    return id < 0 ? -1 : (int64_t)id * a.pool.page_size + (t - p * a.pool.page_size);
}

// First unit of CTA c's share.
__device__ __forceinline__ int64_t share_start(int64_t c, int64_t units, int64_t ctas)
{
    return c * units / ctas;
}

// The walk of a share: segments of consecutive tiles of one row and group.
// The next row's length is fetched a segment ahead.
struct Walk {
    int64_t left;
    int r, g, t;
    Row row;
};

struct Seg {
    Row row;
    int r, g, t0, t1, tiles;
};

__device__ __forceinline__ bool next_seg(const AttnArgs &a, Walk &w, Seg &s)
{
    if (w.left <= 0)
        return false;
    s.row = w.row;
    s.r = w.r;
    s.g = w.g;
    s.t0 = w.t;
    s.tiles = tiles_of(w.row.n);
    s.t1 = (int)min((int64_t)s.tiles, w.t + w.left);
    w.left -= s.t1 - s.t0;
    w.t = s.t1;
    if (s.t1 == s.tiles) {
        w.t = 0;
        if (++w.g == a.groups) {
            w.g = 0;
            ++w.r;
            if (w.left > 0)
                w.row = row_of(a, w.r);
        }
    }
    return true;
}

template <int N>
struct Cfg {
    static constexpr int Q_BYTES = kChunks * N * 128;
    static constexpr int P_BYTES = N * 128;  // 64 tokens a head row
    static constexpr int OFF_Q = 2 * kStageBytes;
    static constexpr int OFF_P = OFF_Q + Q_BYTES;
    static constexpr int OFF_MAX = OFF_P + P_BYTES;     // [4][N] floats
    static constexpr int OFF_HEAD = OFF_MAX + 16 * N;   // [N] floats
    static constexpr int OFF_VALID = OFF_HEAD + 4 * N;  // [2][8] uint16
    static constexpr int OFF_BAR = OFF_VALID + 32;
    static constexpr int BARS = 15;
    static constexpr int OFF_MISC = OFF_BAR + 8 * BARS;  // tmem base, abort, start place
    static constexpr int BYTES = OFF_MISC + 40;
    static constexpr int SMEM = BYTES + 1024;  // the base is aligned to 1024 in the kernel
    static constexpr int COL_S = 4 * N;        // two S^T buffers behind O^T
    static constexpr int TM_COLS = 8 * N;      // 6 N, rounded up to a power of two
    static constexpr int PART = kLatent * N + 2 * N;  // floats of a partial result
};

__device__ __forceinline__ uint32_t tile_unit(uint32_t stage, int chunk, int key, int unit)
{
    return stage + chunk * kChunkBytes + key * 128 + ((unit ^ (key & 7)) << 4);
}

// Four e4m3 codes to bf16 times 2^(scale - 127).  A code's bits placed at
// bf16's sign, low exponent and high mantissa bits are its value times 2^-120,
// subnormal codes included; the multiplier carries the 2^120.
__device__ __forceinline__ uint2 widen4(uint32_t w, __nv_bfloat162 mul)
{
    const uint32_t lo = __byte_perm(w, 0, 0x1404), hi = __byte_perm(w, 0, 0x3424);
    uint32_t a = (lo & 0x80008000u) | ((lo >> 4) & 0x07f007f0u);
    uint32_t b = (hi & 0x80008000u) | ((hi >> 4) & 0x07f007f0u);
    const __nv_bfloat162 x = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&a), mul);
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&b), mul);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&x),
                      *reinterpret_cast<const uint32_t *>(&y));
}

__device__ __forceinline__ uint32_t bf16_pair_of_bits(uint32_t b)
{
    return b | b << 16;
}

__device__ __forceinline__ uint32_t scale_pair(uint32_t w, uint32_t mul)
{
    const __nv_bfloat162 x = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&w),
                                     *reinterpret_cast<__nv_bfloat162 *>(&mul));
    return *reinterpret_cast<const uint32_t *>(&x);
}

// Sixteen codes of one key (latents 16 u .. 16 u + 15) into a stage.  Lanes
// of odd chunks store their second half first, so eight neighbouring lanes
// cover all the banks.
__device__ __forceinline__ void put_codes(uint32_t stage, int key, int u, const uint4 &c,
                                          uint32_t scale)
{
    // 2^(scale - 7): bf16's exponent field holds it up to 2^127
    const uint32_t field = min(scale + 120u, 254u);
    uint32_t m = bf16_pair_of_bits(scale == 255u ? 0x7fc0u : field << 7);
    const __nv_bfloat162 mul = *reinterpret_cast<__nv_bfloat162 *>(&m);
    uint2 v[4] = {widen4(c.x, mul), widen4(c.y, mul), widen4(c.z, mul), widen4(c.w, mul)};
    if (__any_sync(0xffffffffu, scale > 134u)) {
        // what the first multiplier could not hold
        const uint32_t rest =
            bf16_pair_of_bits((scale > 134u && scale < 255u ? scale - 134u + 127u : 127u) << 7);
        #pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = make_uint2(scale_pair(v[i].x, rest), scale_pair(v[i].y, rest));
    }
    const int chunk = u >> 2, unit = 2 * (u & 3), odd = chunk & 1;
    const uint4 h0 = make_uint4(v[0].x, v[0].y, v[1].x, v[1].y);
    const uint4 h1 = make_uint4(v[2].x, v[2].y, v[3].x, v[3].y);
    const uint4 a = odd ? h1 : h0, b = odd ? h0 : h1;
    st_shared_v4(tile_unit(stage, chunk, key, unit + odd), a.x, a.y, a.z, a.w);
    st_shared_v4(tile_unit(stage, chunk, key, unit + 1 - odd), b.x, b.y, b.z, b.w);
}

// A loading warp's place in the share: its tokens of the next tile.
struct Feed {
    Walk w;
    Seg s;
    int t;
    bool live;
};

__device__ __forceinline__ void feed_start(const AttnArgs &a, Feed &f, const Walk &w)
{
    f.w = w;
    f.live = next_seg(a, f.w, f.s);
    f.t = f.live ? f.s.t0 : 0;
}

// The slot of token k of the feed's tile; kNoSlot past the row's end.
constexpr int64_t kNoSlot = INT64_MIN;

__device__ __forceinline__ int64_t feed_slot(const AttnArgs &a, Feed &f, int k, bool lane_on)
{
    int64_t slot = kNoSlot;
    const int t = f.t * kTile + k;
    if (f.live && lane_on && t < f.s.row.n)
        slot = slot_of(a, f.s.row, t);
    return slot;
}

__device__ __forceinline__ void feed_next(const AttnArgs &a, Feed &f)
{
    if (f.live && ++f.t == f.s.t1) {
        f.live = next_seg(a, f.w, f.s);
        f.t = f.s.t0;
    }
}

// Page byte and offset of a slot (-1: no token), telling of bad slots.
__device__ __forceinline__ int64_t place_slot(const AttnArgs &a, int64_t slot, int *off)
{
    int64_t pb = -1;
    *off = 0;
    if (slot == kNoSlot)
        return -1;
    if (!slot_place(a.pool, slot, &pb, off)) {
        atomicOr(a.status, kDevBadPage);
        return -1;
    }
    return pb;
}

// Feed of the loading warps' codes and scales: bypass L1, nothing is read twice.
__device__ __forceinline__ uint4 ld_stream16(const uint8_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// What a loading warp holds of a tile of 8-bit tokens: eight token rows (lane
// u: latents 16 u ..), their rotated elements (eight lanes a token) and their
// scales (four lanes a token, two each).
struct Codes {
    uint4 row[8];
    uint4 rope[2];
    uint32_t scales;
};

__device__ __forceinline__ int64_t shfl64(int64_t v, int src)
{
    return __shfl_sync(0xffffffffu, v, src);
}

__device__ __forceinline__ uint4 load_row8(const AttnArgs &a, int64_t pb, int off, int j, int lane)
{
    const int64_t p = shfl64(pb, j);
    const int o = __shfl_sync(0xffffffffu, off, j);
    return p >= 0 ? ld_stream16(a.pool.base + p + (int64_t)o * kLatent + 16 * lane)
                  : make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ uint4 load_rope8(const AttnArgs &a, int64_t pb, int off, int i, int lane)
{
    const int64_t p = shfl64(pb, 4 * i + (lane >> 3));
    const int o = __shfl_sync(0xffffffffu, off, 4 * i + (lane >> 3));
    return p >= 0 ? ld_stream16(a.pool.base + p + (int64_t)a.pool.page_size * kLatent +
                                (int64_t)o * 2 * kLatRope + 16 * (lane & 7))
                  : make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ uint32_t load_scales8(const AttnArgs &a, int64_t pb, int off, int lane)
{
    const int64_t p = shfl64(pb, lane >> 2);
    const int o = __shfl_sync(0xffffffffu, off, lane >> 2);
    return p >= 0 ? *reinterpret_cast<const uint16_t *>(
                        a.pool.base + p + (int64_t)a.pool.page_size * (kLatent + 2 * kLatRope) +
                        (int64_t)o * kLatGroups + 2 * (lane & 3))
                  : 0x7f7fu;
}

template <int N, bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
    latent_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const AttnArgs a)
{
    using C = Cfg<N>;
    constexpr int NH = N / 8;           // fragments of eight heads
    constexpr int WPT = FP8 ? 8 : 4;    // loading warps of a tile
    constexpr int KPW = kTile / WPT;    // tokens a loading warp brings
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *full = bar, *empty = bar + 2, *s_full = bar + 4, *s_empty = bar + 6;
    uint64_t *q_full = bar + 8, *q_empty = bar + 9, *p_full = bar + 10, *p_empty = bar + 11;
    uint64_t *o_full = bar + 12, *drain = bar + 13;  // drain[2]: the MMA warps' last commits
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    float *smax = reinterpret_cast<float *>(smem + C::OFF_MAX);
    float *shead = reinterpret_cast<float *>(smem + C::OFF_HEAD);
    uint16_t *valid = reinterpret_cast<uint16_t *>(smem + C::OFF_VALID);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], WPT);
            mbar_init(&empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], kSoftWarps);
            mbar_init(&drain[i], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(p_full, kSoftWarps);
        mbar_init(p_empty, 1);
        mbar_init(o_full, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
    }
    if (warp == kWarpPV) {
        tmem_alloc(misc, C::TM_COLS);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_launch_dependents();

    // this CTA's share: a prefix sum of the rows' tiles over the threads
    const int chunk = (a.R + kThreads - 1) / kThreads;
    const int r0 = min(a.R, tid * chunk), r1 = min(a.R, r0 + chunk);
    int64_t mine = 0;
    for (int r = r0; r < r1; ++r)
        mine += tiles_of(row_of(a, r).n);
    int64_t upto = mine;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        upto += lane >= o ? v : 0;
    }
    int64_t *wsum = reinterpret_cast<int64_t *>(smax);
    if (lane == 31)
        wsum[warp] = upto;
    __syncthreads();
    int64_t total = 0, before = upto - mine;
    for (int i = 0; i < kThreads / 32; ++i) {
        total += wsum[i];
        before += i < warp ? wsum[i] : 0;
    }
    const int64_t units = total * a.groups;
    const int64_t ctas = min((int64_t)gridDim.x, units);
    const int c = blockIdx.x;
    const int64_t u0 = c < ctas ? share_start(c, units, ctas) : units;
    const int64_t left = c < ctas ? share_start(c + 1, units, ctas) - u0 : 0;
    int4 *place = reinterpret_cast<int4 *>(a.ws_place);
    if (left > 0 && u0 >= before * a.groups && u0 < (before + mine) * a.groups) {
        int64_t p = before * a.groups;
        int r = r0, tl = tiles_of(row_of(a, r).n);
        while (u0 >= p + (int64_t)tl * a.groups) {
            p += (int64_t)tl * a.groups;
            tl = tiles_of(row_of(a, ++r).n);
        }
        const int g = (int)((u0 - p) / tl), t = (int)((u0 - p) % tl);
        misc[2] = r;
        misc[3] = g;
        misc[4] = t;
        place[c] = make_int4(r, g, t, 0);
    }
    if (left == 0 && tid == 0)
        place[c] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    Walk w;
    w.left = left;
    w.r = misc[2];
    w.g = misc[3];
    w.t = misc[4];
    if (left > 0)
        w.row = row_of(a, w.r);
    Seg s;

    if (warp < kSoftWarps) {
        // ------------------------------------------------ softmax, epilogue
        const int g8 = lane >> 2, c2 = 2 * (lane & 3);
        const int key0 = 16 * warp + g8;  // and key0 + 8
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const uint32_t p_addr = sbase + C::OFF_P;
        const float sl = a.scale_log2;
        int i = 0, k = 0;
        for (; next_seg(a, w, s); ++k) {
            float m[2 * NH], l[2 * NH];
            #pragma unroll
            for (int e = 0; e < 2 * NH; ++e) {
                m[e] = -INFINITY;
                l[e] = 0.0f;
            }
            for (int t = s.t0; t < s.t1; ++t, ++i) {
                const int st = i & 1;
                const uint32_t ph = (i >> 1) & 1;
                // after an abort the waits return at once and the loops run
                // out: every barrier below is still reached by all
                (void)mbar_wait(&full[st], ph, abort_flag, a.status);
                (void)mbar_wait(&s_full[st], ph, abort_flag, a.status);
                __syncwarp();
                tc_fence_after();
                uint32_t sr[4 * NH];
                tmem_ld_16x256b<NH>(tmem + lanes + C::COL_S + st * N, sr);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&s_empty[st]);
                float x[4 * NH];
                #pragma unroll
                for (int e = 0; e < 4 * NH; ++e)
                    x[e] = __uint_as_float(sr[e]);
                const bool v0 = valid[8 * st + key0 % WPT] >> (key0 / WPT) & 1;
                const bool v1 = valid[8 * st + key0 % WPT] >> ((key0 + 8) / WPT) & 1;
                if (!(v0 && v1)) {
                    #pragma unroll
                    for (int j = 0; j < NH; ++j) {
                        x[4 * j] = v0 ? x[4 * j] : -INFINITY;
                        x[4 * j + 1] = v0 ? x[4 * j + 1] : -INFINITY;
                        x[4 * j + 2] = v1 ? x[4 * j + 2] : -INFINITY;
                        x[4 * j + 3] = v1 ? x[4 * j + 3] : -INFINITY;
                    }
                }
                // heads 8 j + c2 + e are entries 2 j + e of m and l
                bool over = false;
                #pragma unroll
                for (int e = 0; e < 2 * NH; ++e) {
                    const int q = 4 * (e >> 1) + (e & 1);
                    over |= fmaf(fmaxf(x[q], x[q + 2]), sl, -m[e]) > kLazy;
                }
                if (named_bar_or(1, 32 * kSoftWarps, over)) {
                    #pragma unroll
                    for (int e = 0; e < 2 * NH; ++e) {
                        const int q = 4 * (e >> 1) + (e & 1);
                        float v = fmaxf(x[q], x[q + 2]);
                        #pragma unroll
                        for (int o = 4; o < 32; o <<= 1)
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
                        if (g8 == 0)
                            smax[warp * N + 8 * (e >> 1) + c2 + (e & 1)] = v;
                    }
                    named_bar_sync(1, 32 * kSoftWarps);
                    #pragma unroll
                    for (int e = 0; e < 2 * NH; ++e) {
                        const int h = 8 * (e >> 1) + c2 + (e & 1);
                        const float top = fmaxf(fmaxf(smax[h], smax[N + h]),
                                                fmaxf(smax[2 * N + h], smax[3 * N + h]));
                        const float nm = fmaxf(m[e], top * sl);
                        const float al = nm == m[e] ? 1.0f : ex2(m[e] - nm);
                        m[e] = nm;
                        l[e] *= al;
                        if (warp == 0 && g8 == 0)
                            shead[h] = al;
                    }
                    if (t > s.t0) {
                        // O^T of the row so far, once its last product is in
                        (void)mbar_wait(p_empty, (i - 1) & 1, abort_flag, a.status);
                        named_bar_sync(1, 32 * kSoftWarps);
                        tc_fence_after();
                        #pragma unroll 1
                        for (int q = 0; q < 4 * N; q += 16) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16(tmem + lanes + q, o);
                            tmem_ld_wait();
                            #pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) *
                                                       shead[q % N + e]);
                            tmem_st_32x32b_x16(tmem + lanes + q, o);
                        }
                        tmem_st_wait();
                    }
                }
                #pragma unroll
                for (int e = 0; e < 2 * NH; ++e) {
                    const int q = 4 * (e >> 1) + (e & 1);
                    const float nm = m[e] == -INFINITY ? 0.0f : -m[e];
                    x[q] = ex2(fmaf(x[q], sl, nm));
                    x[q + 2] = ex2(fmaf(x[q + 2], sl, nm));
                    l[e] += x[q] + x[q + 2];
                }
                // P^T as bf16 (half a step of 2^-8 a weight), head rows of 64
                // tokens, once the product before has read the last ones
                if (i > 0)
                    (void)mbar_wait(p_empty, (i - 1) & 1, abort_flag, a.status);
                __syncwarp();
                #pragma unroll
                for (int j = 0; j < NH; j += 2) {
                    uint32_t f[4];
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const __nv_bfloat162 v =
                            __floats2bfloat162_rn(x[4 * j + 2 * q], x[4 * j + 2 * q + 1]);
                        f[q] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                    const int row = 8 * (j + (lane >> 4)) + (lane & 7);
                    const int unit = (2 * warp + ((lane >> 3) & 1)) ^ (lane & 7);
                    stmatrix_x4_trans(p_addr + row * 128 + unit * 16, f[0], f[1], f[2], f[3]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_full);
            }
            // ---- the segment's sums, then its O^T
            named_bar_sync(1, 32 * kSoftWarps);
            #pragma unroll
            for (int e = 0; e < 2 * NH; ++e) {
                #pragma unroll
                for (int o = 4; o < 32; o <<= 1)
                    l[e] += __shfl_xor_sync(0xffffffffu, l[e], o);
                const int h = 8 * (e >> 1) + c2 + (e & 1);
                if (g8 == 0) {
                    smax[warp * N + h] = l[e];
                    if (warp == 0)
                        shead[h] = m[e];
                }
            }
            named_bar_sync(1, 32 * kSoftWarps);
            const bool whole = s.t0 == 0 && s.t1 == s.tiles;
            float *part = a.ws_part + (int64_t)(2 * c + (k > 0)) * C::PART;
            const int h0 = s.g * 64;
            if (tid < N) {
                const float sum = smax[tid] + smax[N + tid] + smax[2 * N + tid] + smax[3 * N + tid];
                const float mm = shead[tid];
                if (whole) {
                    shead[tid] = sum == 0.0f ? 0.0f : 1.0f / sum;
                    if (a.lse && h0 + tid < a.H)
                        a.lse[s.r * a.ld_lse + h0 + tid] =
                            sum == 0.0f ? -INFINITY : (mm + log2f(sum)) * kLn2;
                } else {
                    part[kLatent * N + tid] = mm;
                    part[kLatent * N + N + tid] = sum;
                }
            }
            (void)mbar_wait(o_full, k & 1, abort_flag, a.status);
            named_bar_sync(1, 32 * kSoftWarps);
            tc_fence_after();
            #pragma unroll 1
            for (int q = 0; q < 4 * N; q += 16) {
                uint32_t o[16];
                tmem_ld_32x32b_x16(tmem + lanes + q, o);
                tmem_ld_wait();
                const int mt = q / N, hq = q % N;  // latents 128 mt .., heads hq ..
                if (whole) {
                    // neighbouring lanes swap, so each stores two latents of a head
                    const int d = 128 * mt + 32 * warp + (lane & ~1);
                    #pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float y0 = __uint_as_float(o[e]) * shead[hq + e];
                        const float y1 = __uint_as_float(o[e + 1]) * shead[hq + e + 1];
                        const bool odd = lane & 1;
                        const float got = __shfl_xor_sync(0xffffffffu, odd ? y0 : y1, 1);
                        const __nv_bfloat162 v = odd ? __floats2bfloat162_rn(got, y1)
                                                     : __floats2bfloat162_rn(y0, got);
                        const int h = h0 + hq + e + odd;
                        if (h < a.H)
                            *reinterpret_cast<__nv_bfloat162 *>(a.out + s.r * a.ldo_row +
                                                                h * a.ldo_head + d) = v;
                    }
                } else {
                    #pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<uint4 *>(part + (int64_t)((q + e) * 128 + 4 * tid)) =
                            make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
            }
            tc_fence_before();
        }
    } else if (warp < kWarpS) {
        // ------------------------------------------------------ token feed
        Feed f;
        feed_start(a, f, w);
        if constexpr (FP8) {
            const int wl = warp - kSoftWarps;
            const int key = wl + WPT * lane;
            const bool on = lane < KPW;
            int off;
            int64_t pb = place_slot(a, feed_slot(a, f, key, on), &off);
            feed_next(a, f);
            int64_t slot = feed_slot(a, f, key, on);
            Codes cd;
            #pragma unroll
            for (int j = 0; j < KPW; ++j)
                cd.row[j] = load_row8(a, pb, off, j, lane);
            cd.scales = load_scales8(a, pb, off, lane);
            cd.rope[0] = load_rope8(a, pb, off, 0, lane);
            cd.rope[1] = load_rope8(a, pb, off, 1, lane);
            uint32_t ok = __ballot_sync(0xffffffffu, pb >= 0);
            for (int i = 0; i < (int)left; ++i) {
                const int st = i & 1;
                const uint32_t stage = sbase + st * kStageBytes;
                // the next tile's places (its slots were fetched a tile ago)
                pb = place_slot(a, slot, &off);
                feed_next(a, f);
                slot = feed_slot(a, f, key, on);
                if (i >= 2 && !mbar_wait(&empty[st], ((i >> 1) - 1) & 1, abort_flag, a.status))
                    break;
                __syncwarp();
                if (lane == 0)
                    valid[8 * st + wl] = (uint16_t)ok;
                const uint32_t scales = cd.scales;
                cd.scales = load_scales8(a, pb, off, lane);
                // each register is filled for the next tile as soon as it is free
                #pragma unroll
                for (int j = 0; j < KPW; ++j) {
                    const uint32_t both =
                        __shfl_sync(0xffffffffu, scales, 4 * j + (lane >> 3));
                    put_codes(stage, wl + WPT * j, lane, cd.row[j],
                              lane & 4 ? both >> 8 : both & 0xffu);
                    cd.row[j] = load_row8(a, pb, off, j, lane);
                }
                #pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint4 v = cd.rope[q];
                    st_shared_v4(tile_unit(stage, kChunks - 1, wl + WPT * (4 * q + (lane >> 3)),
                                           lane & 7), v.x, v.y, v.z, v.w);
                    cd.rope[q] = load_rope8(a, pb, off, q, lane);
                }
                ok = __ballot_sync(0xffffffffu, pb >= 0);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&full[st]);
            }
        } else {
            // four warps bring the even tiles, four the odd ones, straight
            // into the stage: a group waits for its own copies alone
            const int wl = (warp - kSoftWarps) & 3, st = (warp - kSoftWarps) >> 2;
            const int key = wl + WPT * lane;
            const bool on = lane < KPW;
            const uint32_t stage = sbase + st * kStageBytes;
            if (st == 1)
                feed_next(a, f);
            int64_t slot = feed_slot(a, f, key, on);
            for (int i = st; i < (int)left; i += 2) {
                int off;
                const int64_t pb = place_slot(a, slot, &off);
                feed_next(a, f);
                feed_next(a, f);
                slot = feed_slot(a, f, key, on);
                if (i >= 2 && !mbar_wait(&empty[st], ((i >> 1) - 1) & 1, abort_flag, a.status))
                    break;
                __syncwarp();
                const uint32_t ok = __ballot_sync(0xffffffffu, pb >= 0);
                if (lane == 0)
                    valid[8 * st + wl] = (uint16_t)ok;
                #pragma unroll
                for (int j = 0; j < KPW; ++j) {
                    const int64_t p = shfl64(pb, j);
                    const int o = __shfl_sync(0xffffffffu, off, j);
                    const uint8_t *src =
                        a.pool.base + (p >= 0 ? p + (int64_t)o * kLatBf16TokBytes + 16 * lane : 0);
                    const int k = wl + WPT * j;
                    cp_async16(tile_unit(stage, lane >> 3, k, lane & 7), src, p >= 0);
                    cp_async16(tile_unit(stage, 4 + (lane >> 3), k, lane & 7),
                               p >= 0 ? src + 512 : src, p >= 0);
                }
                #pragma unroll
                for (int q = 0; q < KPW / 4; ++q) {
                    const int j = 4 * q + (lane >> 3);
                    const int64_t p = shfl64(pb, j);
                    const int o = __shfl_sync(0xffffffffu, off, j);
                    const uint8_t *src =
                        a.pool.base + (p >= 0 ? p + (int64_t)o * kLatBf16TokBytes + 2 * kLatent +
                                                    16 * (lane & 7)
                                              : 0);
                    cp_async16(tile_unit(stage, kChunks - 1, wl + WPT * j, lane & 7), src, p >= 0);
                }
                cp_async_wait_all();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&full[st]);
            }
        }
    } else if (warp == kWarpS) {
        // -------------------------------------------- queries, S^T = K Q^T
        const bool one = elect_one();
        const uint32_t id = idesc_bf16(kTile, N, false, false);
        int i = 0, k = 0;
        bool ok = true, q_flying = false;
        for (; ok && next_seg(a, w, s); ++k) {
            if (k > 0 && !mbar_wait(q_empty, (k - 1) & 1, abort_flag, a.status))
                break;
            __syncwarp();
            if (one) {
                mbar_arrive_expect_tx(q_full, C::Q_BYTES);
                #pragma unroll 1
                for (int ch = 0; ch < kChunks; ++ch)
                    tma_load_3d(smem + C::OFF_Q + ch * N * 128, &tm_q, q_full, ch * 128, s.g * 64,
                                s.r);
            }
            __syncwarp();
            q_flying = true;
            if (!mbar_wait(q_full, k & 1, abort_flag, a.status))
                break;
            q_flying = false;
            for (int t = s.t0; t < s.t1; ++t, ++i) {
                const int st = i & 1;
                const uint32_t ph = (i >> 1) & 1;
                ok = mbar_wait(&full[st], ph, abort_flag, a.status) &&
                     (i < 2 || mbar_wait(&s_empty[st], ph ^ 1, abort_flag, a.status));
                if (!ok)
                    break;
                __syncwarp();
                tc_fence_after();
                if (one) {
                    const uint32_t ka = sbase + st * kStageBytes, qa = sbase + C::OFF_Q;
                    #pragma unroll 1
                    for (int ch = 0; ch < kChunks; ++ch) {
                        #pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f16(tmem + C::COL_S + st * N,
                                    make_smem_desc(ka + ch * kChunkBytes + kk * 32, 16, 1024,
                                                   kLayoutSw128),
                                    make_smem_desc(qa + ch * N * 128 + kk * 32, 16, 1024,
                                                   kLayoutSw128),
                                    id, ch + kk > 0 ? 1u : 0u);
                    }
                    mma_commit(&s_full[st]);
                    if (t + 1 == s.t1)
                        mma_commit(q_empty);
                }
                __syncwarp();
            }
        }
        if (*abort_flag) {
            if (one)
                mma_commit(&drain[0]);
            __syncwarp();
            if (q_flying)
                (void)mbar_wait_drain(q_full, k & 1);
            (void)mbar_wait_drain(&drain[0], 0);
        }
    } else {
        // --------------------------------------------- O^T += K^T P^T
        const bool one = elect_one();
        const uint32_t id = idesc_bf16(128, N, true, false);
        int i = 0;
        bool ok = true;
        while (ok && next_seg(a, w, s)) {
            for (int t = s.t0; t < s.t1; ++t, ++i) {
                const int st = i & 1;
                ok = mbar_wait(p_full, i & 1, abort_flag, a.status);
                if (!ok)
                    break;
                __syncwarp();
                tc_fence_after();
                if (one) {
                    const uint32_t va = sbase + st * kStageBytes, pa = sbase + C::OFF_P;
                    #pragma unroll 1
                    for (int mt = 0; mt < 4; ++mt) {
                        #pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f16(tmem + mt * N,
                                    make_smem_desc(va + 2 * mt * kChunkBytes + kk * 2048,
                                                   kChunkBytes, 1024, kLayoutSw128),
                                    make_smem_desc(pa + kk * 32, 16, 1024, kLayoutSw128), id,
                                    t > s.t0 || kk > 0 ? 1u : 0u);
                    }
                    mma_commit(&empty[st]);
                    mma_commit(p_empty);
                    if (t + 1 == s.t1)
                        mma_commit(o_full);
                }
                __syncwarp();
            }
        }
        if (*abort_flag) {
            if (one)
                mma_commit(&drain[1]);
            __syncwarp();
            (void)mbar_wait_drain(&drain[1], 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpPV)
        tmem_dealloc(tmem, C::TM_COLS);
}

// Joins the partial results of a row that several shares hold: the CTAs of
// boundary c (blockIdx.x + 1) act if it is the first that cuts its (row,
// group), the shares before and after it holding the pieces.  Threads: 128
// latents x 2 of the group's quads of heads.
constexpr int kJoinThreads = 256;

template <int N>
__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(const AttnArgs a)
{
    using C = Cfg<N>;
    pdl_wait();
    pdl_launch_dependents();
    const int4 *place = reinterpret_cast<const int4 *>(a.ws_place);
    const int c = blockIdx.x + 1, ctas = gridDim.x + 1;
    const int4 here = place[c], prev = place[c - 1];
    const bool prev_same = prev.x == here.x && prev.y == here.y;
    if (here.x < 0 || here.z == 0 || (prev_same && prev.z > 0))
        return;
    int pieces = 0;  // shares c, c + 1, .. that hold more of the row
    for (int b = c; b < ctas; b += kJoinThreads) {
        const int q = b + (int)threadIdx.x;
        bool more = false;
        if (q < ctas) {
            const int4 p = place[q];
            more = p.x == here.x && p.y == here.y && p.z > 0;
        }
        pieces += __syncthreads_count(more);
    }
    const int d = threadIdx.x & 127, mt = blockIdx.y & 3;
    const int quad = 2 * (blockIdx.y >> 2) + (threadIdx.x >> 7);
    // the first piece is the share's first segment if that began with it
    const float *first = a.ws_part + (int64_t)(2 * (c - 1) + !prev_same) * C::PART;
    const float *rest = a.ws_part + (int64_t)2 * c * C::PART;
    const int at = (mt * N + 4 * quad) * 128 + 4 * d;
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    #pragma unroll 4
    for (int q = 0; q <= pieces; ++q) {
        const float *p = q == 0 ? first : rest + (int64_t)(q - 1) * 2 * C::PART;
        const float4 v = *reinterpret_cast<const float4 *>(p + kLatent * N + 4 * quad);
        top[0] = fmaxf(top[0], v.x);
        top[1] = fmaxf(top[1], v.y);
        top[2] = fmaxf(top[2], v.z);
        top[3] = fmaxf(top[3], v.w);
    }
    #pragma unroll
    for (int e = 0; e < 4; ++e)
        top[e] = top[e] == -INFINITY ? 0.0f : top[e];
    float acc[4] = {}, sum[4] = {};
    #pragma unroll 4
    for (int q = 0; q <= pieces; ++q) {
        const float *p = q == 0 ? first : rest + (int64_t)(q - 1) * 2 * C::PART;
        const float4 v = *reinterpret_cast<const float4 *>(p + at);
        const float4 m = *reinterpret_cast<const float4 *>(p + kLatent * N + 4 * quad);
        const float4 l = *reinterpret_cast<const float4 *>(p + kLatent * N + N + 4 * quad);
        const float vv[4] = {v.x, v.y, v.z, v.w}, mm[4] = {m.x, m.y, m.z, m.w};
        const float ll[4] = {l.x, l.y, l.z, l.w};
        #pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float wt = ex2(mm[e] - top[e]);
            acc[e] = fmaf(wt, vv[e], acc[e]);
            sum[e] = fmaf(wt, ll[e], sum[e]);
        }
    }
    const int h0 = here.y * 64 + 4 * quad;
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (h0 + e >= a.H)
            break;
        reinterpret_cast<__nv_bfloat16 *>(a.out)[here.x * a.ldo_row + (h0 + e) * a.ldo_head +
                                                 128 * mt + d] =
            __float2bfloat16(sum[e] == 0.0f ? 0.0f : acc[e] / sum[e]);
        if (a.lse && mt == 0 && d == 0)
            a.lse[here.x * a.ld_lse + h0 + e] =
                sum[e] == 0.0f ? -INFINITY : (top[e] + log2f(sum[e])) * kLn2;
    }
}

int head_columns(int H)
{
    return H <= 16 ? 16 : H <= 32 ? 32 : 64;
}

size_t place_bytes()
{
    return ((size_t)sm_count() * sizeof(int4) + 255) / 256 * 256;
}

template <int N, bool FP8>
idx_status launch_attn(const CUtensorMap &tm, const AttnArgs &a, int ctas, cudaStream_t s)
{
    using C = Cfg<N>;
    static_assert(C::SMEM <= 227 * 1024, "shared memory of a CTA");
    auto kern = latent_attn_kernel<N, FP8>;
    static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return IDX_ERR_CUDA;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
            cudaSuccess)
            return IDX_ERR_CUDA;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaError_t e = launch_pdl(kern, dim3(ctas), dim3(kThreads), C::SMEM, s, tm, a);
    if (e == cudaSuccess && ctas > 1)
        e = launch_pdl(latent_join_kernel<N>, dim3(ctas - 1, 4 * (N / 8)), dim3(kJoinThreads), 0, s,
                       a);
    return launch_status(e);
}

idx_status check_attn(const uint16_t *q, int64_t ldq_row, int64_t ldq_head, int H, int L,
                      int rope_dim, float scale, const uint16_t *out, int64_t ldo_row,
                      int64_t ldo_head, const float *lse, int64_t ld_lse)
{
    if (!q || !out || ldq_head < (int64_t)L + rope_dim || ldq_row < 0 || ldo_head < L ||
        ldo_row < 0 || !(scale > 0.0f) || !(scale <= 3.4e38f) || (lse && ld_lse < H))
        return IDX_ERR_INVALID_ARG;
    if (L != kLatent || rope_dim != kLatRope || H > kMaxHeads || !aligned16(q) ||
        !aligned16(out) || ldq_row % 8 != 0 || ldq_head % 8 != 0 || ldo_row % 8 != 0 ||
        ldo_head % 8 != 0)
        return IDX_ERR_UNSUPPORTED;
    return IDX_OK;
}

// most: an upper bound of the rows' tiles together.
idx_status run_attn(AttnArgs &a, const uint16_t *q, int64_t ldq_row, int64_t ldq_head,
                    idx_latent_format fmt, int64_t most, void *ws, size_t ws_bytes,
                    cudaStream_t s)
{
    if (!ws || !aligned16(ws) || ws_bytes < idx_latent_attention_workspace_size(a.R, a.H))
        return IDX_ERR_WORKSPACE;
    a.status = device_status_ptr();
    if (!a.status)
        return IDX_ERR_CUDA;
    const int n = head_columns(a.H);
    a.groups = (a.H + n - 1) / n;
    a.ws_place = ws;
    a.ws_part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + place_bytes());
    const int ctas = (int)std::min<int64_t>(sm_count(), most * a.groups);
    CUtensorMap tm;
    // bytes of a head row, heads, rows; a stride over one element is free
    const uint64_t dims[3] = {2 * kLatTok, (uint64_t)a.H, (uint64_t)a.R};
    const uint64_t str[2] = {(uint64_t)(a.H > 1 ? 2 * ldq_head : 2 * kLatTok),
                             (uint64_t)(a.R > 1 ? 2 * ldq_row : 2 * kLatTok)};
    const uint32_t box[3] = {128, (uint32_t)n, 1};
    if (!encode_tma_u8(&tm, 3, q, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
        return IDX_ERR_UNSUPPORTED;
    const bool fp8 = fmt == IDX_LATENT_FP8_E4M3;
    switch (n) {
    case 16: return fp8 ? launch_attn<16, true>(tm, a, ctas, s) : launch_attn<16, false>(tm, a, ctas, s);
    case 32: return fp8 ? launch_attn<32, true>(tm, a, ctas, s) : launch_attn<32, false>(tm, a, ctas, s);
    default: return fp8 ? launch_attn<64, true>(tm, a, ctas, s) : launch_attn<64, false>(tm, a, ctas, s);
    }
}

} // namespace
} // namespace idx

using namespace idx;

extern "C" size_t idx_latent_attention_workspace_size(int R, int H)
{
    if (R <= 0 || H <= 0)
        return 0;
    const int n = head_columns(H);
    return place_bytes() + (size_t)2 * sm_count() * (kLatent * n + 2 * n) * sizeof(float);
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
    idx_status ok = check_attn(q, ldq_row, ldq_head, H, L, rope_dim, scale, out, ldo_row,
                               ldo_head, lse, ld_lse);
    if (ok == IDX_OK)
        ok = check_pool(kv_pages, page_stride_bytes, num_pages, page_size, fmt);
    if (ok != IDX_OK)
        return ok;
    AttnArgs a = {};
    a.pool = make_pool(kv_pages, page_stride_bytes, num_pages, page_size);
    a.slots = slots;
    a.indptr = indptr;
    a.num_slots = num_slots;
    a.next_n = 1;
    a.R = R;
    a.H = H;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.ldo_row = ldo_row;
    a.ldo_head = ldo_head;
    a.lse = lse;
    a.ld_lse = ld_lse;
    return run_attn(a, q, ldq_row, ldq_head, fmt, num_slots / kTile + R, ws, ws_bytes,
                    (cudaStream_t)stream);
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
    idx_status ok = check_attn(q, ldq_row, ldq_head, H, L, rope_dim, scale, out,
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
    a.block_table = block_table;
    a.bt_stride = bt_stride;
    a.context_lens = context_lens;
    a.ctx_per_row = ctx_per_row;
    a.next_n = next_n;
    a.max_len = max_model_len;
    a.R = B * next_n;
    a.H = H;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.ldo_row = ldo_row;
    a.ldo_head = ldo_head;
    a.lse = lse;
    a.ld_lse = ld_lse;
    const int64_t row_tiles = std::max(1, (int)(((int64_t)max_model_len + kTile - 1) / kTile));
    return run_attn(a, q, ldq_row, ldq_head, fmt, row_tiles * a.R, ws, ws_bytes,
                    (cudaStream_t)stream);
}
