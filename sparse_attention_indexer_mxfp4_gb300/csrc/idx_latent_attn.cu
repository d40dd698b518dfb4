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
// the heads on its N: 16, 32 or 64 columns a CTA, so few heads waste no tensor
// work, the running sums O^T stay in tensor memory for a row's whole length
// (4 N columns), and the tile is read in place both times, K-major by its
// token rows and M-major by its latent columns (the same 128-byte swizzled
// rows describe both).  In the paged form the heads of several rows of a
// sequence share the columns (each row with its own end), so their tokens are
// read once.  What 64 columns do not hold is further groups; the CTAs of one
// share's groups run side by side and find each other's tokens in L2.
//
// Work is split over the flat list of (row, tile): every share is an equal
// contiguous part, whatever the rows' lengths (a row: a ragged row, or a
// sequence of the paged form).  A row counts a few tiles more than it has: what
// a CTA that begins it pays for the end of the row before.  Rows that lie in one
// share are finished there; the others leave unnormalised sums with their
// maximum in scratch and a second kernel joins them in share order.
//
// What bounds it: with 64 columns shared memory's data path.  Of 3600 cycles a
// tile of 8-bit tokens the products' operands take 1920 wavefronts (36 x 32 and
// 16 x 48), loads, stores and shuffles 1930 (the counters overlap a little):
// 2048 rows x 64 heads x 2048 slots 802 us, 728 TFLOP/s, the tensor pipe 47 %
// busy.  With 16 columns it is the same path (1300 and 1590 of 2920 cycles) and
// DRAM beside it: 32 contexts of 4 to 32 thousand 8-bit tokens 107 us, 3.8 TB/s.
// Bf16 tokens need no widening: four contexts of 100 to 131 thousand, 32 columns,
// 102 us with the joining kernel, 5.6 TB/s while this one runs.  Few rows wait:
// about 9 thousand cycles until a CTA has its first tokens, twice a table and
// then what it names.
//
// Warps: 0-3 softmax and epilogue; 4-11 bring tokens in (slot -> page ->
// global loads; 8-bit codes are widened to bf16 on the way, exactly, by moving
// their bits and a multiplication with a power of two); 12 loads queries and
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
constexpr int kSoftWarps = 4;
constexpr int kFeedWarps = 4;              // loading warps of a tile
constexpr int kToks = kTile / kFeedWarps;  // tokens each brings
constexpr int kLoadWarps = 2 * kFeedWarps; // even tiles, odd tiles
constexpr int kWarpS = kSoftWarps + kLoadWarps, kWarpPV = kWarpS + 1;
constexpr int kThreads = (kWarpPV + 1) * 32;
constexpr int kMaxHeads = 128;
constexpr float kLazy = 40.0f;  // a score may exceed its running maximum by 2^40
constexpr float kFinite = 3.4028234e38f;
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

struct AttnArgs {
    LatentPool pool;
    const int32_t *slots, *indptr;  // ragged rows (indptr null: paged)
    int num_slots;
    const int32_t *block_table, *context_lens;
    int64_t bt_stride;
    int ctx_per_row, max_len;
    int rows, next;            // rows of the list; query rows in each (paged: next_n)
    int H, groups, hgroups;    // head groups, times groups of query rows
    int hpg, rpg;              // heads and query rows of a group's columns
    int charge;                // tiles a row counts besides its own
    uint32_t inv_hpg;          // column / hpg = column * inv_hpg >> 16
    float scale_log2;  // scale * log2(e)
    uint16_t *out;
    int64_t ldo_row, ldo_head;
    float *lse;
    int64_t ld_lse;
    // By row (by_row), or by the share that begins the row: the row, that share,
    // its pieces (fewer than two: whole), whether a segment lies before it.
    int4 *ws_cut;
    int by_row;
    int uncut;       // shares end with rows: no partial results
    float *ws_part;  // two segments a CTA: O^T, then maxima, then sums
    int page_stride;  // pool.stride in 32 bits: one multiplication
    unsigned int *status;
};

// Where a row's tokens are listed, and how many it has (paged: the most any
// of its query rows sees).
struct Row {
    int64_t first;
    int n;
};

// Paged: how many tokens query row j of sequence b sees.
__device__ __forceinline__ int query_end(const AttnArgs &a, int b, int j)
{
    const int end = a.ctx_per_row ? a.context_lens[b * a.next + j]
                                  : a.context_lens[b] - a.next + j + 1;
    return min(max(end, 0), a.max_len);
}

// Out of line: every role asks, once a row.
__device__ __noinline__ Row row_of(const AttnArgs &a, int r)
{
    if (a.indptr) {
        const int lo = min(max(a.indptr[r], 0), a.num_slots);
        const int hi = min(max(a.indptr[r + 1], 0), a.num_slots);
        return {lo, max(0, hi - lo)};
    }
    int n = query_end(a, r, a.next - 1);
    if (a.ctx_per_row)
        #pragma unroll 1
        for (int j = 0; j + 1 < a.next; ++j)
            n = max(n, query_end(a, r, j));
    return {r * a.bt_stride, n};
}

// A row without tokens still takes one (empty) tile: it has outputs.
__device__ __forceinline__ int tiles_of(int n)
{
    return n > kTile ? (n + kTile - 1) / kTile : 1;
}

// A group's first query row and head.
struct Group {
    int j0, h0;
};

__device__ __forceinline__ Group group_of(const AttnArgs &a, int g)
{
    const int q = g / a.hgroups;
    return {q * a.rpg, (g - q * a.hgroups) * a.hpg};
}

// Query row (within the list's row) and head of a group's column; false for a
// column that has none.
__device__ __forceinline__ bool column_place(const AttnArgs &a, const Group &g, int col, int *j,
                                             int *h)
{
    const int q = (int)(col * a.inv_hpg >> 16);
    *j = g.j0 + q;
    *h = g.h0 + col - q * a.hpg;
    return q < a.rpg && *j < a.next && *h < a.H;
}

// The walk of a share: segments of consecutive tiles of one row.  The next
// row's length is fetched a segment ahead.
struct Walk {
    int left;
    int r, t;
    Row row;
};

struct Seg {
    Row row;
    int r, t0, t1, tiles;
};

__device__ __forceinline__ bool next_seg(const AttnArgs &a, Walk &w, Seg &s)
{
    if (w.left <= 0)
        return false;
    s.row = w.row;
    s.r = w.r;
    s.t0 = w.t;
    s.tiles = tiles_of(w.row.n);
    s.t1 = min(s.tiles, w.t + w.left);
    w.left -= s.t1 - s.t0;
    w.t = s.t1;
    if (s.t1 == s.tiles) {
        w.t = 0;
        ++w.r;
        if (w.left > 0)
            w.row = row_of(a, w.r);
    }
    return true;
}

// Reduces each of CNT values over the eight lanes that differ in bits 2-4,
// halving the values a lane carries at every step (CNT - 1 exchanges, not 3
// CNT).  Steps are instances of their own: as a loop whose count halves, the
// values went through local memory (64 columns 3 % slower).  Lane l is left with CNT / 8 results (one, for fewer than eight) in
// v[0 ..]; returns which value v[0] is.
template <int O, int CNT, int SIZE, typename Op>
__device__ __forceinline__ int reduce_step(float (&v)[SIZE], int lane, Op op)
{
    if constexpr (O < 4) {
        return 0;
    } else if constexpr (CNT > 1) {
        constexpr int H = CNT / 2;
        const bool up = lane & O;
        #pragma unroll
        for (int e = 0; e < H; ++e) {
            const float got = __shfl_xor_sync(0xffffffffu, up ? v[e] : v[e + H], O);
            v[e] = op(up ? v[e + H] : v[e], got);
        }
        return (up ? H : 0) + reduce_step<O / 2, H>(v, lane, op);
    } else {
        v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], O));
        return reduce_step<O / 2, 1>(v, lane, op);
    }
}

template <int CNT, typename Op>
__device__ __forceinline__ int reduce_rows(float (&v)[CNT], int lane, Op op)
{
    return reduce_step<16, CNT>(v, lane, op);
}

template <int N>
struct Cfg {
    static constexpr int Q_BYTES = kChunks * N * 128;
    // 64 tokens a head row; the epilogue turns 1 KB a warp over in it, twice
    static constexpr int P_BYTES = 8192;
    static_assert(N <= 64, "a head row is 128 bytes");
    static constexpr int OFF_Q = 2 * kStageBytes;
    static constexpr int OFF_P = OFF_Q + Q_BYTES;
    static constexpr int OFF_MAX = OFF_P + P_BYTES;     // [4][N] floats
    static constexpr int OFF_HEAD = OFF_MAX + 16 * N;   // [N] floats
    static constexpr int OFF_END = OFF_HEAD + 4 * N;    // [N] int
    static constexpr int OFF_VALID = OFF_END + 4 * N;   // [2][8] uint16
    static constexpr int OFF_BAR = OFF_VALID + 32;
    static constexpr int BARS = 19;
    static constexpr int OFF_MISC = OFF_BAR + 8 * BARS;  // tmem base, abort, start place
    static constexpr int BYTES = OFF_MISC + 40;
    static constexpr int SMEM = BYTES + 1024;  // the base is aligned to 1024 in the kernel
    static constexpr int COL_S = 4 * N;        // two S^T buffers behind O^T
    static constexpr int TM_COLS = 8 * N;      // 6 N, rounded up to a power of two
    static constexpr int PART = kLatent * N + 2 * N;  // floats of a partial result
};

// Four e4m3 codes to bf16 times `mul`.  A code's bits placed at bf16's sign,
// low exponent and high mantissa bits (two bytes: s0000eee emmm0000) are its
// value times 2^-120, subnormal codes included; the multiplier carries 2^120.
// A NaN code (all seven bits set) becomes 480 times its scale, which no other
// code is: nan_codes finds it, fix_codes mends it.
__device__ __forceinline__ uint2 widen4(uint32_t w, uint32_t mul)
{
    const uint32_t hi = (w & 0x80808080u) | ((w >> 4) & 0x07070707u);
    const uint32_t lo = (w << 4) & 0xf0f0f0f0u;
    uint32_t a = __byte_perm(lo, hi, 0x5140), b = __byte_perm(lo, hi, 0x7362);
    const __nv_bfloat162 m = *reinterpret_cast<__nv_bfloat162 *>(&mul);
    const __nv_bfloat162 x = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&a), m);
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&b), m);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&x),
                      *reinterpret_cast<const uint32_t *>(&y));
}

// Has a byte's top bit set where one of four codes is a NaN (a carry out of
// 0xff may set the next byte's too): adding one turns the sign of seven ones.
// Two instructions a word in put_codes: 64 columns 2.7 % slower, 16 columns 3.3;
// before the wait for the stage, 2.4 and 5.2.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w)
{
    return (w + 0x01010101u) ^ w;
}

// An e8m0 scale as the multiplier of widen4: 2^(scale - 7) twice, up to 2^127
// (scale 134); fix_codes does the rest.
constexpr uint32_t kPlainScale = 134;

__device__ __forceinline__ uint32_t widen_mul(uint32_t scale)
{
    return min(scale, kPlainScale) * 0x00800080u + 120u * 0x00800080u;
}

// The slots' tokens of nothing: what a loading warp reads for a place without
// a token.
__device__ uint4 g_no_token[kLatBf16TokBytes / 16];

// A loading warp's place in the share: tile t of a row of which the share
// holds the tiles before `end`, and the tiles left after them.
struct Feed {
    Row row;
    int r, t, end, left;
};

__device__ __forceinline__ void feed_row(Feed &f)
{
    f.end = min(tiles_of(f.row.n), f.t + f.left);
    f.left -= f.end - f.t;
}

__device__ __forceinline__ void feed_next(const AttnArgs &a, Feed &f)
{
    if (++f.t < f.end)
        return;
    f.t = f.end = 0;
    f.row.n = 0;
    if (f.left > 0) {
        f.row = row_of(a, ++f.r);
        feed_row(f);
    }
}

// A token on its way: what its table holds (a slot, or a page's id) and, for
// the paged form, its offset in the page.  The entry is only fetched here;
// place_of, a tile later, is the first to look at it.
struct Entry {
    int32_t id;
    int off;  // -1: no token (past the row's end, or another lane's)
};

__device__ __forceinline__ Entry feed_entry(const AttnArgs &a, const Feed &f, int k, bool lane_on)
{
    Entry e = {0, -1};
    const int t = f.t * kTile + k;
    if (lane_on && t < f.row.n) {
        const int32_t *at = a.slots + f.row.first + t;
        e.off = 0;
        if (!a.indptr) {
            const int p = page_of(a.pool, t);
            e.off = t - p * a.pool.page_size;
            at = a.block_table + f.row.first + p;
        }
        e.id = *at;
    }
    return e;
}

// Page byte and offset of an entry (-1: no token), telling of bad ones.
__device__ __forceinline__ int64_t place_of(const AttnArgs &a, const Entry &e, int *off)
{
    if (e.off < 0)
        return -1;
    *off = e.off;
    int page = e.id;
    if (a.indptr) {
        page = page_of(a.pool, e.id);
        *off = e.id - page * a.pool.page_size;
    }
    if (e.id >= 0 && page < a.pool.num_pages)
        return (int64_t)page * a.page_stride;
    atomicOr(a.status, kDevBadPage);
    return -1;
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

__device__ __forceinline__ const uint8_t *shfl_ptr(const uint8_t *p, int src)
{
    return reinterpret_cast<const uint8_t *>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), src));
}

// The kToks tokens that a loading warp brings of a tile: token i of warp w is
// the tile's key 2 kFeedWarps (i / 2) + 2 w + i % 2, and lane i holds its place.
// Pairs of keys that differ in the lowest bit are handled together: eight
// lanes at a time reach all banks, and every shared address is a constant of
// the lane plus a constant.
struct Places {
    const uint8_t *row, *rope, *scale;  // lanes below kToks
    uint32_t ok;                        // which of the tokens exist
};

template <bool FP8>
__device__ __forceinline__ Places places_of(const AttnArgs &a, const Entry &e)
{
    int off;
    const int64_t pb = place_of(a, e, &off);
    Places p;
    p.ok = __ballot_sync(0xffffffffu, pb >= 0);
    p.row = p.rope = p.scale = reinterpret_cast<const uint8_t *>(g_no_token);
    if (pb >= 0) {
        const uint8_t *page = a.pool.base + pb;
        if (FP8) {
            p.row = page + (int64_t)off * kLatent;
            page += (int64_t)a.pool.page_size * kLatent;
            p.rope = page + (int64_t)off * (2 * kLatRope);
            page += (int64_t)a.pool.page_size * (2 * kLatRope);
            p.scale = page + (int64_t)off * kLatGroups;
        } else {
            p.row = page + (int64_t)off * kLatBf16TokBytes;
            p.rope = p.row + 2 * kLatent;
        }
    }
    return p;
}

// 8-bit tokens on their way through registers.  Lane: key bit (lane / 4) % 2,
// chunks lane / 8 and 4 more, sixteen codes at 16 (lane % 4) of each.
struct Codes {
    uint4 row[kToks / 2][2];  // pairs of tokens, halves of the latents
    uint4 rope[kToks / 4];    // eight lanes a token
    uint32_t scales;          // lane 2 i + half: that half's four scales of token i
};

__device__ __forceinline__ void load_codes(const Places &p, int lane, Codes &c)
{
    c.scales = *reinterpret_cast<const uint32_t *>(shfl_ptr(p.scale, (lane >> 1) & (kToks - 1)) +
                                                   4 * (lane & 1));
    const int at = 64 * (lane >> 3) + 16 * (lane & 3);
    #pragma unroll
    for (int j = 0; j < kToks / 2; ++j) {
        const uint8_t *src = shfl_ptr(p.row, 2 * j + ((lane >> 2) & 1)) + at;
        c.row[j][0] = ld_stream16(src);
        c.row[j][1] = ld_stream16(src + 256);
    }
    #pragma unroll
    for (int q = 0; q < kToks / 4; ++q)
        c.rope[q] = ld_stream16(shfl_ptr(p.rope, 4 * q + (lane >> 3)) + 16 * (lane & 7));
}

constexpr int kPairBytes = 2 * kFeedWarps * 128;  // between a warp's pairs of keys

// Shared address of this lane's codes of pair 0 in its first chunk (the second
// sixteen bytes are at ^ 16), and of its rotated elements.
__device__ __forceinline__ uint32_t codes_at(uint32_t stage, int wl, int lane)
{
    const int k = 2 * wl + ((lane >> 2) & 1);
    return stage + (lane >> 3) * kChunkBytes + k * 128 + (((2 * (lane & 3)) ^ (k & 7)) << 4);
}

__device__ __forceinline__ uint32_t rope_at(uint32_t stage, int wl, int lane)
{
    const int k = 2 * wl + ((lane >> 3) & 1);
    return stage + (kChunks - 1) * kChunkBytes + (2 * kFeedWarps * (lane >> 4) + k) * 128 +
           (((lane & 7) ^ (k & 7)) << 4);
}

// Half h (chunks 4 h .., the rotated elements with the second) as bf16 into
// the stage.  Returns whether one of the lane's codes is a NaN.
__device__ __forceinline__ bool put_codes(uint32_t stage, int wl, int lane, Codes &c, int h)
{
    const uint32_t u0 = codes_at(stage, wl, lane), u1 = u0 ^ 16, half = h * 4 * kChunkBytes;
    uint32_t nan = 0;
    #pragma unroll
    for (int j = 0; j < kToks / 2; ++j) {
        const uint32_t four =
            __shfl_sync(0xffffffffu, c.scales, 4 * j + 2 * ((lane >> 2) & 1) + h);
        const uint32_t mul = widen_mul(__byte_perm(four, 0, 0x4440 | (lane >> 3)));
        const uint4 v = c.row[j][0];
        c.row[j][0] = c.row[j][1];  // the second half's turn: one code for both
        nan |= nan_codes(v.x) | nan_codes(v.y) | nan_codes(v.z) | nan_codes(v.w);
        const uint2 a = widen4(v.x, mul), b = widen4(v.y, mul);
        const uint2 d = widen4(v.z, mul), e = widen4(v.w, mul);
        st_shared_v4(u0 + half + j * kPairBytes, a.x, a.y, b.x, b.y);
        st_shared_v4(u1 + half + j * kPairBytes, d.x, d.y, e.x, e.y);
    }
    if (h != 0) {
        const uint32_t ur = rope_at(stage, wl, lane);
        #pragma unroll
        for (int q = 0; q < kToks / 4; ++q)
            st_shared_v4(ur + 2 * q * kPairBytes, c.rope[q].x, c.rope[q].y, c.rope[q].z,
                         c.rope[q].w);
    }
    return (nan & 0x80808080u) != 0;
}

// Scales over 2^7 and the NaN scale: multiplies the warp's own part of the
// stage by what widen_mul left out (latents beyond 57344).  NaN codes: makes
// NaN of what widen4 made of them, 480 = 1.875 * 2^8 times the scale so far.
// Both are rare.
__device__ __noinline__ void fix_codes(uint32_t stage, int wl, int lane, uint32_t scales, int h)
{
    #pragma unroll 1
    for (int j = 0; j < kToks / 2; ++j) {
        const uint32_t four =
            __shfl_sync(0xffffffffu, scales, 4 * j + 2 * ((lane >> 2) & 1) + h);
        const uint32_t s = four >> (8 * (lane >> 3)) & 0xffu;
        const uint32_t nan = ((min(s, kPlainScale) + 8u) << 7 | 0x70u) * 0x00010001u;
        const uint32_t bits = s == 255u         ? 0x7fc0u
                              : s > kPlainScale ? (s - kPlainScale + 127u) << 7
                                                : 0x3f80u;
        uint32_t mul = bits | bits << 16;
        const __nv_bfloat162 m = *reinterpret_cast<__nv_bfloat162 *>(&mul);
        #pragma unroll 1
        for (int e = 0; e < 2; ++e) {
            const uint32_t to =
                (codes_at(stage, wl, lane) ^ (16 * e)) + j * kPairBytes + h * 4 * kChunkBytes;
            uint32_t v[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(to));
            for (int q = 0; q < 4; ++q) {
                v[q] |= __vcmpeq2(v[q] & 0x7fff7fffu, nan) & 0x7fff7fffu;
                const __nv_bfloat162 y = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&v[q]), m);
                v[q] = *reinterpret_cast<const uint32_t *>(&y);
            }
            st_shared_v4(to, v[0], v[1], v[2], v[3]);
        }
    }
}

// The same halves of bf16 tokens, straight into the stage.
__device__ __forceinline__ void copy_tokens(uint32_t stage, int wl, int lane, const Places &p,
                                            int h)
{
    #pragma unroll
    for (int i = 0; i < kToks; ++i) {
        const int k = 2 * kFeedWarps * (i >> 1) + 2 * wl + (i & 1);
        cp_async16(stage + (4 * h + (lane >> 3)) * kChunkBytes + k * 128 +
                       (((lane & 7) ^ (k & 7)) << 4),
                   shfl_ptr(p.row, i) + 512 * h + 16 * lane);
    }
    if (h == 0)
        return;
    const uint32_t ur = rope_at(stage, wl, lane);
    #pragma unroll
    for (int q = 0; q < kToks / 4; ++q)
        cp_async16(ur + 2 * q * kPairBytes, shfl_ptr(p.rope, 4 * q + (lane >> 3)) + 16 * (lane & 7));
}

// A tile's tokens from `from` on, which some column is not to see, and the
// latents of one lane of O^T (128 mt + tid): zeros in place of what is not
// finite, since a weight of zero does not hide it.  Byte mt of the result is
// the first such token (64: none).
__device__ __noinline__ uint32_t hide_tokens(uint8_t *stage, int from, int tid)
{
    uint32_t first = kTile * 0x01010101u;
    #pragma unroll 1
    for (int k = kTile - 1; k >= from; --k)
        #pragma unroll 1
        for (int mt = 0; mt < 4; ++mt) {
            const int d = 128 * mt + tid;
            uint16_t *at = reinterpret_cast<uint16_t *>(
                stage + (d >> 6) * kChunkBytes + k * 128 + (((d >> 3 & 7) ^ (k & 7)) << 4) +
                2 * (d & 7));
            if ((*at & 0x7f80u) == 0x7f80u) {
                *at = 0;
                first = (first & ~(0xffu << 8 * mt)) | (uint32_t)k << 8 * mt;
            }
        }
    return first;
}

// Once the tile's product is in O^T: NaN in the columns that see such a token
// (end: each column's, counted from the tile's first token).
template <int N>
__device__ __noinline__ void show_tokens(uint32_t o_lanes, uint32_t first, const int *end, int tile0)
{
    #pragma unroll 1
    for (int q = 0; q < 4 * N; q += 16) {
        const int k = first >> 8 * (q / N) & 0xffu;
        if (!__any_sync(0xffffffffu, k < kTile))
            continue;
        uint32_t o[16];
        tmem_ld_32x32b_x16(o_lanes + q, o);
        tmem_ld_wait();
        #pragma unroll
        for (int e = 0; e < 16; ++e)
            o[e] = k < min(end[q % N + e] - tile0, kTile) ? 0x7fffffffu : o[e];
        tmem_st_32x32b_x16(o_lanes + q, o);
    }
    tmem_st_wait();
}

// SHARED: rows of a sequence share its tokens, each up to its own end (paged,
// next > 1).  The others go without that code: the prefill chunk's 2048 rows
// 810 us, with it 831; 64 rows 49.2, with it 50.2.
template <int N, bool FP8, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
    latent_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const AttnArgs a)
{
    using C = Cfg<N>;
    constexpr int NH = N / 8;           // fragments of eight heads
    constexpr int KEPT = 2 * NH > 8 ? NH / 4 : 1;  // what reduce_rows leaves a lane
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    // full, empty [2 stage + half]: a stage's chunks 0-3, and the rest
    uint64_t *full = bar, *empty = bar + 4, *s_full = bar + 8, *s_empty = bar + 10;
    uint64_t *q_full = bar + 12, *q_empty = bar + 13, *p_full = bar + 14, *p_empty = bar + 15;
    uint64_t *o_full = bar + 16, *drain = bar + 17;  // drain[2]: the MMA warps' last commits
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    float *smax = reinterpret_cast<float *>(smem + C::OFF_MAX);
    float *shead = reinterpret_cast<float *>(smem + C::OFF_HEAD);
    uint16_t *valid = reinterpret_cast<uint16_t *>(smem + C::OFF_VALID);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&full[i], kFeedWarps);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
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

    // this CTA's share: a prefix sum of the rows' tiles, and what each row
    // counts besides, over the threads
    const int chunk = (a.rows + kThreads - 1) / kThreads;
    const int r0 = min(a.rows, tid * chunk), r1 = min(a.rows, r0 + chunk);
    // Rows of an ascending list have at most INT32_MAX / 4 tiles and two charges
    // each together; one that descends can name its slots any number of times.
    constexpr uint32_t kTooMany = INT32_MAX;
    const auto plus = [](uint32_t x, uint32_t y) { return min(x + y, kTooMany); };
    uint32_t own = 0;
    #pragma unroll 1
    for (int r = r0; r < r1; ++r)
        own = plus(own, tiles_of(row_of(a, r).n) + a.charge);
    const int mine = own;
    uint32_t upto = own;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
        upto = plus(upto, lane >= o ? v : 0);
    }
    int *wsum = reinterpret_cast<int *>(smax);
    if (lane == 31)
        wsum[warp] = upto;
    __syncthreads();
    uint32_t all = 0, lower = upto - own;
    #pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        all = plus(all, wsum[i]);
        lower = plus(lower, i < warp ? wsum[i] : 0);
    }
    const bool too_many = all == kTooMany;  // no CTA has a share
    const int total = too_many ? 1 : all, before = lower;
    // equal shares, the first ones a tile longer
    const Group group = group_of(a, blockIdx.x);
    const int p = blockIdx.y, shares = min((int)gridDim.y, total);
    const int each = total / shares, more = total - each * shares;
    // the share's bounds as places in the list and as tiles (a place within a
    // row's charge is its first tile)
    #pragma unroll 1
    for (int e = 0; e < 2; ++e) {
        const int u = (p + e) * each + min(p + e, more);
        if (p + e <= shares && u >= before && u < before + mine) {
            int q = before, r = r0, n = mine;  // of one row, usually
            if (chunk > 1) {
                n = tiles_of(row_of(a, r).n) + a.charge;
                #pragma unroll 1
                while (u >= q + n) {
                    q += n;
                    n = tiles_of(row_of(a, ++r).n) + a.charge;
                }
            }
            int t = max(0, u - q - a.charge);
            if (a.uncut && u > q) {
                // the share that the row begins in has all of it
                q += n;
                ++r;
                t = 0;
            }
            misc[2 + e] = q - r * a.charge + t;
            if (e == 0) {
                misc[4] = r;
                misc[5] = t;
            }
        }
    }
    if (!a.by_row && !a.uncut && blockIdx.x == 0 && tid == 0)
        a.ws_cut[p] = make_int4(-1, 0, 0, 0);
    if (too_many && blockIdx.x == 0 && p == 0) {
        if (tid == 0)
            atomicOr(a.status, kDevBadBounds);
        if (a.by_row && !a.uncut && tid < a.rows)  // fewer than SMs
            a.ws_cut[tid] = make_int4(-1, 0, 0, 0);
    }
    __syncthreads();
    const int tiles1 = p + 1 < shares ? (int)misc[3] : total - a.rows * a.charge;
    const int left = p < shares && !too_many ? tiles1 - (int)misc[2] : 0;
    if (a.hpg * a.rpg < N) {
        // columns without a head: their query rows are zeros
        #pragma unroll 1
        for (int e = tid; e < C::Q_BYTES / 16; e += kThreads)
            st_shared_v4(sbase + C::OFF_Q + 16 * e, 0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    __syncthreads();
    tc_fence_after();
    // one value for the warp, as the compiler sees it too
    const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);
    Walk w = {left, 0, 0, {0, 0}};  // a CTA without a share has an empty walk
    if (left > 0) {
        w.r = misc[4];
        w.t = misc[5];
        w.row = row_of(a, w.r);
    }
    Seg s;

    if (warp < kSoftWarps) {
        // ------------------------------------------------ softmax, epilogue
        const int g8 = lane >> 2, c2 = 2 * (lane & 3);
        const int key0 = 16 * warp + g8;  // and key0 + 8
        const int *send = reinterpret_cast<const int *>(smem + C::OFF_END);
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
            // each column's end; before the first of them nothing is masked
            int first_end = INT_MAX;
            if constexpr (SHARED) {
                if (tid < N) {
                    int j, h;
                    reinterpret_cast<int *>(smem + C::OFF_END)[tid] =
                        column_place(a, group, tid, &j, &h) ? query_end(a, s.r, j) : s.row.n;
                }
                #pragma unroll 1
                for (int j = 0; j < a.rpg; ++j)
                    first_end = min(first_end, query_end(a, s.r, min(group.j0 + j, a.next - 1)));
                named_bar_sync(1, 32 * kSoftWarps);
            }
            #pragma unroll 1
            for (int t = s.t0; t < s.t1; ++t, ++i) {
                const int st = i & 1;
                const uint32_t ph = (i >> 1) & 1;
                // after an abort the waits return at once and the loops run
                // out: every barrier below is still reached by all
                (void)mbar_wait(&full[2 * st], ph, abort_flag, a.status);
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
                const auto exists = [&](int key) {
                    const int pair = key / (2 * kFeedWarps), in = key % (2 * kFeedWarps);
                    return (valid[8 * st + (in >> 1)] >> (2 * pair + (in & 1)) & 1) != 0;
                };
                const bool v0 = exists(key0), v1 = exists(key0 + 8);
                if (!(v0 && v1)) {
                    #pragma unroll
                    for (int j = 0; j < NH; ++j) {
                        x[4 * j] = v0 ? x[4 * j] : -INFINITY;
                        x[4 * j + 1] = v0 ? x[4 * j + 1] : -INFINITY;
                        x[4 * j + 2] = v1 ? x[4 * j + 2] : -INFINITY;
                        x[4 * j + 3] = v1 ? x[4 * j + 3] : -INFINITY;
                    }
                }
                [[maybe_unused]] uint32_t hidden = kTile * 0x01010101u;  // of hide_tokens
                if (SHARED && (t + 1) * kTile > first_end) {
                    // a token that is not finite has no finite score
                    bool odd = false;
                    #pragma unroll
                    for (int e = 0; e < 2 * NH; ++e) {
                        const int lim = send[8 * (e >> 1) + c2 + (e & 1)] - t * kTile;
                        const int q = 4 * (e >> 1) + (e & 1);
                        odd |= v0 && key0 >= lim && !(fabsf(x[q]) <= kFinite);
                        odd |= v1 && key0 + 8 >= lim && !(fabsf(x[q + 2]) <= kFinite);
                        x[q] = key0 < lim ? x[q] : -INFINITY;
                        x[q + 2] = key0 + 8 < lim ? x[q + 2] : -INFINITY;
                    }
                    if (named_bar_or(1, 32 * kSoftWarps, odd)) {
                        (void)mbar_wait(&full[2 * st + 1], ph, abort_flag, a.status);
                        hidden = hide_tokens(smem + st * kStageBytes, max(0, first_end - t * kTile),
                                             tid);
                        __syncwarp();
                    }
                }
                // heads 8 j + c2 + e are entries 2 j + e of m and l
                if (t == s.t0) {
                    // the reference of each head begins as its first token's
                    // score: it only has to be within range of the others
                    if (warp == 0 && g8 == 0) {
                        #pragma unroll
                        for (int e = 0; e < 2 * NH; ++e)
                            shead[8 * (e >> 1) + c2 + (e & 1)] = x[4 * (e >> 1) + (e & 1)];
                    }
                    named_bar_sync(1, 32 * kSoftWarps);
                    #pragma unroll
                    for (int e = 0; e < 2 * NH; ++e)
                        m[e] = shead[8 * (e >> 1) + c2 + (e & 1)] * sl;
                }
                bool over = false;
                #pragma unroll
                for (int e = 0; e < 2 * NH; ++e) {
                    const int q = 4 * (e >> 1) + (e & 1);
                    over |= fmaf(fmaxf(x[q], x[q + 2]), sl, -m[e]) > kLazy;
                }
                if (named_bar_or(1, 32 * kSoftWarps, over)) {
                    float v[2 * NH];
                    #pragma unroll
                    for (int e = 0; e < 2 * NH; ++e) {
                        const int q = 4 * (e >> 1) + (e & 1);
                        v[e] = fmaxf(x[q], x[q + 2]);
                    }
                    const int b = reduce_rows(v, lane, [](float y, float z) { return fmaxf(y, z); });
                    #pragma unroll
                    for (int e = 0; e < KEPT; ++e)
                        smax[warp * N + 8 * ((b + e) >> 1) + c2 + ((b + e) & 1)] = v[e];
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
                if (SHARED && (t + 1) * kTile > first_end &&
                    __any_sync(0xffffffffu, hidden != kTile * 0x01010101u)) {
                    (void)mbar_wait(p_empty, i & 1, abort_flag, a.status);
                    __syncwarp();
                    tc_fence_after();
                    show_tokens<N>(tmem + lanes, hidden, send, t * kTile);
                }
            }
            // ---- the segment's sums, then its O^T
            named_bar_sync(1, 32 * kSoftWarps);
            const int b = reduce_rows(l, lane, [](float y, float z) { return y + z; });
            #pragma unroll
            for (int e = 0; e < KEPT; ++e)
                smax[warp * N + 8 * ((b + e) >> 1) + c2 + ((b + e) & 1)] = l[e];
            if (warp == 0 && g8 == 0) {
                #pragma unroll
                for (int e = 0; e < 2 * NH; ++e)
                    shead[8 * (e >> 1) + c2 + (e & 1)] = m[e];
            }
            named_bar_sync(1, 32 * kSoftWarps);
            const bool whole = s.t0 == 0 && s.t1 == s.tiles;
            float *part = a.ws_part +
                          (int64_t)(2 * (p * a.groups + (int)blockIdx.x) + (k > 0)) * C::PART;
            int *at_col = reinterpret_cast<int *>(smem + C::OFF_END);  // whole: places in out
            if (tid < N) {
                const float sum = smax[tid] + smax[N + tid] + smax[2 * N + tid] + smax[3 * N + tid];
                const float mm = shead[tid];
                if (whole) {
                    shead[tid] = sum == 0.0f ? 0.0f : 1.0f / sum;
                    int j, h;
                    const bool is = column_place(a, group, tid, &j, &h);
                    at_col[tid] = is ? (int)((j * a.ldo_row + h * a.ldo_head) >> 3) : -1;
                    if (is && a.lse)
                        a.lse[((int64_t)s.r * a.next + j) * a.ld_lse + h] =
                            sum == 0.0f ? -INFINITY : (mm + log2f(sum)) * kLn2;
                } else {
                    part[kLatent * N + tid] = mm;
                    part[kLatent * N + N + tid] = sum;
                }
                if (tid == 0 && blockIdx.x == 0 && s.t0 == 0 && !a.uncut && (a.by_row || !whole)) {
                    // the shares that hold the rest: `more - p - 1` longer ones first
                    const int rest = s.tiles - s.t1, longer = max(0, more - p - 1);
                    const int in = min(rest, longer * (each + 1));
                    a.ws_cut[a.by_row ? s.r : p] = make_int4(
                        s.r, p, 1 + (in + each) / (each + 1) + (rest - in + each - 1) / each, k > 0);
                }
            }
            (void)mbar_wait(o_full, k & 1, abort_flag, a.status);
            named_bar_sync(1, 32 * kSoftWarps);
            tc_fence_after();
            if (whole) {
                // 32 latents (this warp's) x 16 heads at a time, turned over in
                // the warp's part of the P buffer (free: the last product is in)
                // so that four lanes store 64 bytes of a head
                const uint32_t turn0 = p_addr + warp * 2048;
                uint16_t *to = a.out + (int64_t)s.r * a.next * a.ldo_row + 32 * warp +
                               8 * (lane & 3);
                #pragma unroll 2
                for (int q = 0; q < 4 * N; q += 16) {
                    const uint32_t turn = turn0 + (q & 16) * 64;
                    uint32_t o[2][8];
                    tmem_ld_16x256b<2>(tmem + lanes + q, o[0]);
                    tmem_ld_16x256b<2>(tmem + lanes + (16u << 16) + q, o[1]);
                    tmem_ld_wait();
                    const int hq = q % N;
                    uint32_t f[2][4];  // eight heads each: latents 8 i ..
                    #pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 inv =
                            *reinterpret_cast<const float2 *>(shead + hq + 8 * e + c2);
                        #pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const __nv_bfloat162 v = __floats2bfloat162_rn(
                                __uint_as_float(o[i >> 1][4 * e + 2 * (i & 1)]) * inv.x,
                                __uint_as_float(o[i >> 1][4 * e + 2 * (i & 1) + 1]) * inv.y);
                            f[e][i] = *reinterpret_cast<const uint32_t *>(&v);
                        }
                    }
                    __syncwarp();
                    // head rows of 64 bytes, 16-byte pieces rotated against bank conflicts
                    #pragma unroll
                    for (int e = 0; e < 2; ++e)
                        stmatrix_x4_trans(turn + (8 * e + (lane & 7)) * 64 +
                                              (((lane >> 3) ^ ((lane >> 1) & 3)) << 4),
                                          f[e][0], f[e][1], f[e][2], f[e][3]);
                    __syncwarp();
                    #pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = 8 * e + (lane >> 2);
                        uint4 v;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                     : "r"(turn + row * 64 +
                                           (((lane & 3) ^ ((row >> 1) & 3)) << 4)));
                        const int off = at_col[hq + row];
                        if (off >= 0)
                            *reinterpret_cast<uint4 *>(to + ((int64_t)off << 3) + 128 * (q / N)) =
                                v;
                    }
                }
            } else {
                #pragma unroll 1
                for (int q = 0; q < 4 * N; q += 32) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(tmem + lanes + q, o);
                    tmem_ld_wait();
                    #pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4 *>(part + (int64_t)((q + e) * 128 + 4 * tid)) =
                            make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
            }
            named_bar_sync(1, 32 * kSoftWarps);  // the next row's columns go where these were
            tc_fence_before();
        }
    } else if (warp < kWarpS) {
        // ------------------------------------------------------ token feed
        // half of the warps bring the even tiles, half the odd ones, so that one
        // group's loads are in flight while the other fills its stage
        const int wl = (warp - kSoftWarps) % kFeedWarps, st = (warp - kSoftWarps) / kFeedWarps;
        const int key = 2 * kFeedWarps * (lane >> 1) + 2 * wl + (lane & 1);
        const bool on = lane < kToks;
        const uint32_t stage = sbase + st * kStageBytes;
        Feed f = {w.row, w.r, w.t, 0, left};
        if (left > 0)
            feed_row(f);
        Entry entry = {0, -1};
        Places pl;
        Codes cd;
        int skip = st;  // tiles to pass over: the other half's
        #pragma unroll 1
        for (int i = st - 4; i < left; i += 2) {
            if (i >= 0) {
                const uint32_t ph = ((i >> 1) - 1) & 1;
                bool ok = true;
                #pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    ok = i < 2 || mbar_wait(&empty[2 * st + h], ph, abort_flag, a.status);
                    if (!ok)
                        break;
                    __syncwarp();
                    if (h == 0 && lane == 0)
                        valid[8 * st + wl] = (uint16_t)pl.ok;
                    if constexpr (FP8) {
                        // in registers since the last tile
                        const bool nan = put_codes(stage, wl, lane, cd, h);
                        if (__any_sync(0xffffffffu,
                                       nan || __vcmpgtu4(cd.scales, kPlainScale * 0x01010101u) != 0)) {
                            __syncwarp();
                            fix_codes(stage, wl, lane, cd.scales, h);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&full[2 * st + h]);
                    } else {
                        copy_tokens(stage, wl, lane, pl, h);
                        cp_async_commit();
                    }
                }
                if (!ok)
                    break;
                if constexpr (!FP8) {
                    cp_async_wait<1>();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&full[2 * st]);
                    cp_async_wait<0>();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&full[2 * st + 1]);
                }
            }
            // the half's next tile (its entries were fetched a tile ago)
            pl = places_of<FP8>(a, entry);
            if (FP8 && i >= st - 2)
                load_codes(pl, lane, cd);
            #pragma unroll 1
            for (; skip > 0; --skip)
                feed_next(a, f);
            skip = 2;
            entry = feed_entry(a, f, key, on);
        }
        if constexpr (!FP8)
            cp_async_wait<0>();  // after an abort
    } else if (warp == kWarpS) {
        // -------------------------------------------- queries, S^T = K Q^T
        const bool one = elect_one();
        const uint32_t id = idesc_bf16(kTile, N, false, false);
        const uint32_t q_bytes = kChunks * a.hpg * a.rpg * 128;
        int i = 0, k = 0;
        bool ok = true, q_flying = false;
        for (; ok && next_seg(a, w, s); ++k) {
            if (k > 0 && !mbar_wait(q_empty, (k - 1) & 1, abort_flag, a.status))
                break;
            __syncwarp();
            if (one) {
                mbar_arrive_expect_tx(q_full, q_bytes);
                #pragma unroll 1
                for (int ch = 0; ch < kChunks; ++ch)
                    tma_load_3d(smem + C::OFF_Q + ch * N * 128, &tm_q, q_full, ch * 128,
                                group.h0, s.r * a.next + group.j0);
            }
            __syncwarp();
            q_flying = true;
            if (!mbar_wait(q_full, k & 1, abort_flag, a.status))
                break;
            q_flying = false;
            #pragma unroll 1
            for (int t = s.t0; t < s.t1; ++t, ++i) {
                const int st = i & 1;
                const uint32_t ph = (i >> 1) & 1;
                ok = i < 2 || mbar_wait(&s_empty[st], ph ^ 1, abort_flag, a.status);
                uint32_t kd = desc_lo(sbase + st * kStageBytes), qd = desc_lo(sbase + C::OFF_Q);
                #pragma unroll 1
                for (int ch = 0; ok && ch < kChunks; ++ch) {
                    if (ch == 0 || ch == 4) {
                        ok = mbar_wait(&full[2 * st + (ch >> 2)], ph, abort_flag, a.status);
                        if (!ok)
                            break;
                        __syncwarp();
                        tc_fence_after();
                    }
                    #pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f16(tmem + C::COL_S + st * N, kd + 2 * kk, qd + 2 * kk, kDescHiSw128,
                                id, kk > 0 ? 1u : (ch > 0 ? 1u : 0u), one);
                    kd += kChunkBytes >> 4;
                    qd += N * 128 >> 4;
                }
                if (!ok)
                    break;
                mma_commit_if(&s_full[st], one);
                mma_commit_if(q_empty, one && t + 1 == s.t1);
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
            #pragma unroll 1
            for (int t = s.t0; t < s.t1; ++t, ++i) {
                const int st = i & 1;
                ok = mbar_wait(p_full, i & 1, abort_flag, a.status);
                if (!ok)
                    break;
                __syncwarp();
                tc_fence_after();
                uint32_t vd = desc_lo(sbase + st * kStageBytes, kChunkBytes);
                const uint32_t pd = desc_lo(sbase + C::OFF_P);
                #pragma unroll 1
                for (int mt = 0; mt < 4; ++mt) {
                    #pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f16(tmem + mt * N, vd + kk * (2048 >> 4), pd + 2 * kk, kDescHiSw128,
                                id, kk > 0 ? 1u : (t > s.t0 ? 1u : 0u), one);
                    vd += 2 * kChunkBytes >> 4;
                    if (mt & 1)
                        mma_commit_if(&empty[2 * st + (mt >> 1)], one);
                }
                mma_commit_if(p_empty, one);
                mma_commit_if(o_full, one && t + 1 == s.t1);
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

// Joins the partial results of a row that several shares hold:
//     out = sum_q 2^(m_q - m) O_q / sum_q 2^(m_q - m) l_q,   m = max_q m_q.
// 64 rows x 64 heads cut into 152 shares: 28 MB through L2, 8.6 us.
// blockIdx.x: the row's entry of ws_cut; blockIdx.y: a quad of columns (MANY:
// and 128 latents); blockIdx.z: the group.  The pieces lie in L2, a thousand
// cycles away or more, so a thread asks for four pieces at once, a thread a
// latent (of all four tiles of them), and where a row has many, four teams of
// threads take four pieces each in turn (one row of 16 heads on 2048 keys 11.0 us
// in all; with eight teams, whose threads have half the registers, 11.7; two
// 14.9).
constexpr int kTeams = 4;

template <int N, bool MANY>
__global__ void __launch_bounds__(MANY ? 128 * kTeams : 128) latent_join_kernel(const AttnArgs a)
{
    using C = Cfg<N>;
    constexpr int MT = MANY ? 1 : 4, TEAMS = MANY ? kTeams : 1;
    __shared__ float4 s_top[TEAMS], s_sum[TEAMS], s_acc[TEAMS][MANY ? 128 : 1];
    pdl_wait();
    pdl_launch_dependents();
    const int4 cut = a.ws_cut[blockIdx.x];
    const int pieces = cut.z;
    if (pieces < 2)
        return;
    const int d = threadIdx.x & 127, team = threadIdx.x >> 7;
    const int quad = MANY ? blockIdx.y >> 2 : blockIdx.y, mt0 = MANY ? blockIdx.y & 3 : 0;
    const int64_t step = (int64_t)2 * a.groups * C::PART;
    // a share leaves its first segment at 2 (share, group), its last after it
    const float *rest = a.ws_part + cut.y * step + (int64_t)blockIdx.z * 2 * C::PART;
    const int at_m = kLatent * N + 4 * quad, at_o = (mt0 * N + 4 * quad) * 128 + 4 * d;
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, sum[4] = {}, acc[MT][4] = {};
    #pragma unroll 1
    for (int q0 = 4 * team; q0 < pieces; q0 += 4 * TEAMS) {
        float4 m[4], l[4], o[4][MT];
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int q = q0 + i;
            const float *f = rest + (q == 0 ? cut.w * C::PART : q * step);
            m[i] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            l[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            #pragma unroll
            for (int x = 0; x < MT; ++x)
                o[i][x] = l[i];
            if (q < pieces) {
                m[i] = *reinterpret_cast<const float4 *>(f + at_m);
                l[i] = *reinterpret_cast<const float4 *>(f + at_m + N);
                #pragma unroll
                for (int x = 0; x < MT; ++x)
                    o[i][x] = *reinterpret_cast<const float4 *>(f + at_o + x * N * 128);
            }
        }
        #pragma unroll
        for (int e = 0; e < 4; ++e) {
            const auto of = [e](const float4 &v) {
                return e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
            };
            const float nt = fmaxf(fmaxf(fmaxf(of(m[0]), of(m[1])), fmaxf(of(m[2]), of(m[3]))), top[e]);
            const float ref = nt == -INFINITY ? 0.0f : nt;
            const float c = ex2(top[e] - ref);
            top[e] = nt;
            sum[e] *= c;
            #pragma unroll
            for (int x = 0; x < MT; ++x)
                acc[x][e] *= c;
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = ex2(of(m[i]) - ref);
                sum[e] = fmaf(w, of(l[i]), sum[e]);
                #pragma unroll
                for (int x = 0; x < MT; ++x)
                    acc[x][e] = fmaf(w, of(o[i][x]), acc[x][e]);
            }
        }
    }
    if constexpr (MANY) {
        s_acc[team][d] = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
        if (d == 0) {
            s_top[team] = make_float4(top[0], top[1], top[2], top[3]);
            s_sum[team] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        }
        __syncthreads();
        if (team > 0)
            return;
        #pragma unroll
        for (int e = 0; e < 4; ++e) {
            top[e] = -INFINITY;
            #pragma unroll
            for (int i = 0; i < TEAMS; ++i)
                top[e] = fmaxf(top[e], reinterpret_cast<const float *>(&s_top[i])[e]);
            const float ref = top[e] == -INFINITY ? 0.0f : top[e];
            sum[e] = acc[0][e] = 0.0f;
            #pragma unroll
            for (int i = 0; i < TEAMS; ++i) {
                const float w = ex2(reinterpret_cast<const float *>(&s_top[i])[e] - ref);
                sum[e] = fmaf(w, reinterpret_cast<const float *>(&s_sum[i])[e], sum[e]);
                acc[0][e] = fmaf(w, reinterpret_cast<const float *>(&s_acc[i][d])[e], acc[0][e]);
            }
        }
    }
    const Group group = group_of(a, blockIdx.z);
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
        int j, h;
        if (!column_place(a, group, 4 * quad + e, &j, &h))
            continue;
        const int64_t r = (int64_t)cut.x * a.next + j;
        __nv_bfloat16 *to = reinterpret_cast<__nv_bfloat16 *>(a.out) + r * a.ldo_row +
                            h * a.ldo_head + 128 * mt0 + d;
        const float inv = sum[e] == 0.0f ? 0.0f : 1.0f / sum[e];
        #pragma unroll
        for (int x = 0; x < MT; ++x)
            to[128 * x] = __float2bfloat16(acc[x][e] * inv);
        if (a.lse && mt0 == 0 && d == 0)
            a.lse[r * a.ld_lse + h] =
                sum[e] == 0.0f ? -INFINITY
                               : ((top[e] == -INFINITY ? 0.0f : top[e]) + log2f(sum[e])) * kLn2;
    }
}

int columns_of(int n)
{
    return n <= 16 ? 16 : n <= 32 ? 32 : 64;
}

size_t cut_bytes()
{
    return ((size_t)sm_count() * sizeof(int4) + 255) / 256 * 256;
}

template <int N, bool FP8, bool SHARED>
idx_status launch_attn(const CUtensorMap &tm, const AttnArgs &a, int shares, cudaStream_t s)
{
    using C = Cfg<N>;
    static_assert(C::SMEM <= 227 * 1024, "shared memory of a CTA");
    auto kern = latent_attn_kernel<N, FP8, SHARED>;
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
    cudaError_t e = launch_pdl(kern, dim3(a.groups, shares), dim3(kThreads), C::SMEM, s, tm, a);
    if (e == cudaSuccess && shares > 1 && !a.uncut) {
        const int entries = a.by_row ? a.rows : shares - 1;
        // Teams up to three blocks of them an SM, one at a time; us with and
        // without: at 2048 keys 16 columns x 4 rows 12.0 and 20.6, 32 columns x 12
        // 19.0 and 20.4, x 16 21.0 and 19.7; 64 columns x 6 20.7 and 24.0, x 10 24.0
        // and 21.1.
        if (entries * N * a.groups <= 3 * sm_count())
            e = launch_pdl(latent_join_kernel<N, true>, dim3(entries, N, a.groups),
                           dim3(128 * kTeams), 0, s, a);
        else
            e = launch_pdl(latent_join_kernel<N, false>, dim3(entries, N / 4, a.groups), dim3(128),
                           0, s, a);
    }
    return launch_status(e);
}

template <int N, bool FP8>
idx_status launch_for(const CUtensorMap &tm, const AttnArgs &a, int shares, cudaStream_t s)
{
    return a.next > 1 ? launch_attn<N, FP8, true>(tm, a, shares, s)
                      : launch_attn<N, FP8, false>(tm, a, shares, s);
}

idx_status check_attn(const uint16_t *q, int64_t ldq_row, int64_t ldq_head, int H, int L,
                      int rope_dim, float scale, const uint16_t *out, int64_t ldo_row,
                      int64_t ldo_head, const float *lse, int64_t ld_lse)
{
    if (!q || !out || ldq_head < (int64_t)L + rope_dim || ldq_row < 0 || ldo_head < L ||
        ldo_row < 0 || !(scale > 0.0f) || !(scale * kLog2e <= 3.4e38f) || (lse && ld_lse < H))
        return IDX_ERR_INVALID_ARG;
    if (L != kLatent || rope_dim != kLatRope || H > kMaxHeads || !aligned16(q) ||
        !aligned16(out) || ldq_row % 8 != 0 || ldq_head % 8 != 0 || ldo_row % 8 != 0 ||
        ldo_head % 8 != 0)
        return IDX_ERR_UNSUPPORTED;
    return IDX_OK;
}

// Groups of columns: `hpg` heads of `rpg` query rows each.
struct Columns {
    int hpg, rpg, hgroups, groups;
};

Columns columns_for(int H, int next)
{
    Columns c;
    // up to 64 heads, and as many query rows of them as 64 hold
    c.hpg = std::min(H, 64);
    c.rpg = std::min(next, 64 / c.hpg);
    c.hgroups = (H + c.hpg - 1) / c.hpg;
    c.groups = c.hgroups * ((next + c.rpg - 1) / c.rpg);
    return c;
}

// Rows of few keys are not cut: up to four tiles a CTA more cost less than
// the joining kernel (7.0 us whole, 8.6 cut, for 4 rows of 64 keys).
constexpr int64_t kUncutKeys = 4 * kTile;

// most: an upper bound of the rows' tiles together; keys: of any row's.
idx_status run_attn(AttnArgs &a, const uint16_t *q, int64_t ldq_row, int64_t ldq_head,
                    idx_latent_format fmt, int64_t most, int64_t keys, void *ws, size_t ws_bytes,
                    cudaStream_t s)
{
    const int R = a.rows * a.next;
    const size_t need = idx_latent_attention_workspace_size(R, a.H, keys);
    if (need > 0 && (!ws || !aligned16(ws) || ws_bytes < need))
        return IDX_ERR_WORKSPACE;
    a.uncut = keys <= kUncutKeys;
    a.status = device_status_ptr();
    if (!a.status)
        return IDX_ERR_CUDA;
    const Columns c = columns_for(a.H, a.next);
    a.hpg = c.hpg;
    a.rpg = c.rpg;
    a.inv_hpg = 65536 / a.hpg + 1;
    a.hgroups = c.hgroups;
    a.groups = c.groups;
    // places in out are kept in units of eight elements, in 32 bits
    const int64_t span = (a.next - 1) * a.ldo_row + (a.H - 1) * a.ldo_head;
    if (a.groups > sm_count() || most > INT32_MAX / 4 || a.pool.stride > INT32_MAX ||
        span / 8 > INT32_MAX)
        return IDX_ERR_UNSUPPORTED;
    a.page_stride = (int)a.pool.stride;
    const int n = columns_of(a.hpg * a.rpg);
    a.ws_cut = static_cast<int4 *>(ws);
    a.ws_part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + cut_bytes());
    // one CTA per SM, the same number for every group
    const int shares =
        (int)std::min<int64_t>(sm_count() / a.groups, most);
    a.by_row = a.rows < shares;
    // The end of a row (its sums, its output, the next row's first scores) costs
    // a CTA about as much as this many tiles: 64 columns 24 rows of 2048 keys
    // 24.1 us (uncharged 27.7), 64 rows 45.4 (47.3).  Shares of one tile are left
    // equal: 8 rows of 512 keys 15.2 us charged, 13.6 uncharged.
    a.charge = most <= shares ? 0 : n == 64 ? 2 : 1;
    CUtensorMap tm;
    // bytes of a head row, heads, rows; a stride over one element is free
    const uint64_t dims[3] = {2 * kLatTok, (uint64_t)a.H, (uint64_t)R};
    const uint64_t str[2] = {(uint64_t)(a.H > 1 ? 2 * ldq_head : 2 * kLatTok),
                             (uint64_t)(R > 1 ? 2 * ldq_row : 2 * kLatTok)};
    const uint32_t box[3] = {128, (uint32_t)a.hpg, (uint32_t)a.rpg};
    if (!encode_tma_u8(&tm, 3, q, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
        return IDX_ERR_UNSUPPORTED;
    const bool fp8 = fmt == IDX_LATENT_FP8_E4M3;
    switch (n) {
    case 16: return fp8 ? launch_for<16, true>(tm, a, shares, s) : launch_for<16, false>(tm, a, shares, s);
    case 32: return fp8 ? launch_for<32, true>(tm, a, shares, s) : launch_for<32, false>(tm, a, shares, s);
    default: return fp8 ? launch_for<64, true>(tm, a, shares, s) : launch_for<64, false>(tm, a, shares, s);
    }
}

} // namespace
} // namespace idx

using namespace idx;

extern "C" size_t idx_latent_attention_workspace_size(int R, int H, int64_t max_keys)
{
    if (R <= 0 || H <= 0 || max_keys <= kUncutKeys)
        return 0;
    // at most a CTA per SM, each with two segments of at most 64 columns (which
    // rows of a sequence share whatever H is)
    const int64_t columns = columns_of((int)std::min<int64_t>(64, (int64_t)R * H));
    return cut_bytes() + (size_t)(2 * sm_count() * (kLatent + 2) * columns) * sizeof(float);
}

extern "C" int idx_latent_attention_launches(int R, int next_n, int H, int64_t max_keys)
{
    if (R <= 0 || next_n <= 0 || H <= 0)
        return 0;
    // rows are cut where a group of columns has two CTAs or more
    return max_keys > kUncutKeys && sm_count() / columns_for(H, next_n).groups > 1 ? 2 : 1;
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
    a.num_slots = (int)std::min<int64_t>(num_slots, INT32_MAX);
    a.rows = R;
    a.next = 1;
    a.H = H;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.ldo_row = ldo_row;
    a.ldo_head = ldo_head;
    a.lse = lse;
    a.ld_lse = ld_lse;
    return run_attn(a, q, ldq_row, ldq_head, fmt, num_slots / kTile + R, num_slots, ws,
                    ws_bytes,
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
    a.next = next_n;
    a.max_len = max_model_len;
    a.rows = B;
    a.H = H;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.ldo_row = ldo_row;
    a.ldo_head = ldo_head;
    a.lse = lse;
    a.ld_lse = ld_lse;
    const int64_t row_tiles = std::max(1, (int)(((int64_t)max_model_len + kTile - 1) / kTile));
    return run_attn(a, q, ldq_row, ldq_head, fmt, row_tiles * B, max_model_len, ws,
                    ws_bytes, (cudaStream_t)stream);
}
