// idx_kv4_attn.cu -- attention of grouped heads over the 4-bit cache, by ragged
// slots or whole paged contexts, and the weights it gives the cached tokens.
//
// For one key head, the columns are the query heads that share it (of all rows
// of a sequence), in blocks of 8 or 16; tokens are the other side:
//
//     S^T [32 tokens x cols] = K [32 x 128] . Q^T,   O^T [128 x cols] += V^T . P^T
//
// What bounds it is reading the cache, 136 bytes a token and head, and widening
// it: 7 TB/s are 47 elements a clock and SM.  So the codes are widened in
// registers, straight into the operand fragments of warp-level products, and
// never pass through shared memory a second time (a widened tile would take 94
// of its 128 bytes a clock to write, and as many to read): tokens are the
// products' 16 rows, so that 8 columns fill an instruction.
//
//  * The hardware's conversion gives a pair of e2m1 as f16, exactly.  Queries
//    become f16 under a power of two of their own, which bf16's 8 bits survive.
//  * A key's scale stands for 32 elements, two product steps: their sum is
//    scaled in 32 bits.
//  * A value's scale goes to the weight: P_g = P 2^(e_g - E_g), E_g the largest
//    exponent met, as f16 pairs (O follows E_g like the running maximum).  Tokens
//    over 2^15 under E_g, and NaN scales, take a second form of the product with
//    bf16 weights, which have an exponent to spare.
//  * Values lie with pairs of elements in a byte, and the product wants pairs of
//    tokens: the nibbles of two tokens change places before they are widened,
//    four instructions for sixteen elements.
//
// Every warp walks 32 tokens of each tile of 128 with a running maximum and sum
// of its own and a ring of its own, filled by asynchronous copies (16 bytes, the
// pieces of a row turned by its number so that fragments are read without bank
// conflicts).  Work is the flat list of (row or sequence, key head, tile); CTAs
// take equal contiguous shares of it and a second kernel joins what they cut.  Few
// units of few tiles go to a cluster of CTAs each instead, which joins its sums through
// its shared memory: no second kernel.  The ring runs on over the ends of a share's
// segments; there the warps hand their sums on in fragments, through the one place of
// the ring that is free.
//
// Measured: 32 contexts of 4096 to 32768 tokens x 8 key heads, 4 columns, 125 us (690
// MB, 0.81 of the copy rate; 0.64 instructions a cycle and scheduler bound it); 4 of 100 to 131
// thousand, 16 columns, 139; 64 rows x 2048 slots x 8 key heads 50 to 57.  Rings filled
// by bulk tensor copies and barriers took 134 and 154 for the first two.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cooperative_groups.h>
#include <float.h>

#include "idx_kv4.cuh"

namespace idx {
namespace {

constexpr int kThreads = 128, kWarps = 4;
constexpr int kSub = 32;                // tokens of a warp's step
constexpr int kTile = kWarps * kSub;    // of a CTA's
constexpr int kSubCodes = kSub * kKv4Codes;
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
constexpr float kLazy = 4.0f;           // a score may exceed its running maximum by 2^4
constexpr int kBias = 10;               // weights are held 2^10 larger: up to 2^14 in f16
constexpr int kScaleUp = 1;             // and scaled values' up to 2 more
constexpr int kScaleRange = 15;         // f16 holds 2 to 2^-14 without loss
// Rows of few keys are not cut: no scratch and no joining kernel.
constexpr int kUncutKeys = 4 * kTile;
// Teams: CTAs of a cluster that share a unit, for up to kTeamTiles tiles a group, and
// kTeamLeast in all.
constexpr int kTeamMost = 8, kTeamTiles = 5, kTeamLeast = 256;
constexpr int kJoinThreads = 256;
constexpr int kJoinFew = 8;  // pieces of a unit that one warp joins

struct Kv4Args {
    const uint16_t *q;
    int64_t ldq_row, ldq_head;
    Kv4Pool pool;
    int group;        // query heads of a key head
    int cols;         // columns of a unit: rows of a sequence x group
    int blocks;       // blocks of columns
    // ragged slots
    const int32_t *slots, *indptr;
    int64_t num_slots;
    // whole contexts
    const int32_t *table;
    int64_t bt_stride;
    const int32_t *ctx;
    int ctx_per_row, next_n, max_len;
    int B;            // rows or sequences
    float scale_log2;
    uint16_t *out;
    int64_t ldo_row, ldo_head;
    float *lse;
    int64_t ld_lse;
    int uncut;        // units are not cut
    int team;         // CTAs that share a unit (0: shares of the list)
    // A unit (a sequence's key head and block of columns) that is begun: sequence, head and
    // block, pieces, and twice the share that has the first, plus one where that is not the
    // share's first segment.  By unit, or where there are more of them than shares by the
    // share that begins a unit and leaves it to the next (none: no pieces).
    int4 *ws_cut;
    int by_unit;
    float *ws_part;   // two segments a share: O, maxima, sums
    unsigned int *status;
    // weights of tokens
    const float *lse_in;
    int64_t ld_lse_in, ld_lse_head;
    const float *mass;
    int64_t ld_batch, ld_head;
    int width;
    float *mass_out;
    int64_t ldo_batch, ldo_mass_head;
};

// ------------------------------------------------------------------- pieces

__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same on sums of zero.
__device__ __forceinline__ void mma16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                            uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ void mma16_bf(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8 x 8 block of 16-bit elements in fragment registers, transposed.
__device__ __forceinline__ uint32_t turn8(uint32_t v)
{
    uint32_t t;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(t) : "r"(v));
    return t;
}

__device__ __forceinline__ uint32_t as_u32(__half2 v)
{
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v)
{
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ __half2 as_h2(uint32_t v)
{
    return *reinterpret_cast<const __half2 *>(&v);
}

__device__ __forceinline__ __nv_bfloat162 as_b2(uint32_t v)
{
    return *reinterpret_cast<const __nv_bfloat162 *>(&v);
}

// f16 pairs that bf16 holds (e2m1 values).
__device__ __forceinline__ uint32_t to_bf16x2(uint32_t h)
{
    const float2 f = __half22float2(as_h2(h));
    return as_u32(__floats2bfloat162_rn(f.x, f.y));
}

// Copies of scattered pieces: 64 bytes are fetched for one and no more (64 rows x
// 64 heads x 2048 slots 56 us, with the usual granularity 71).
__device__ __forceinline__ void cp_async16_alone(uint32_t saddr, const void *src)
{
    asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16;" ::"r"(saddr),
                 "l"(reinterpret_cast<uint64_t>(src))
                 : "memory");
}

__device__ __forceinline__ void cp_async4_alone(uint32_t saddr, const void *src)
{
    asm volatile("cp.async.ca.shared.global.L2::64B [%0], [%1], 4;" ::"r"(saddr),
                 "l"(reinterpret_cast<uint64_t>(src))
                 : "memory");
}

// Loads from shared memory by address, so that what varies is added once a step.
__device__ __forceinline__ uint32_t lds32(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}

__device__ __forceinline__ uint32_t lds16(uint32_t at)
{
    uint16_t v;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(at));
    return v;
}

__device__ __forceinline__ float4 lds128f(uint32_t at)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at));
    return v;
}

// 2^x of a float's exponent field and beyond it (underflow gives 0).
__device__ __forceinline__ float pow2i(int x)
{
    return ex2((float)x);
}

// ------------------------------------------------------------------ the list

// How tokens are found: by slots, by pages of any size, by pages that hold whole
// steps of 32 tokens.
enum Mode { kSlots, kPages, kWholePages };

// A unit's tokens: the longest of its rows.
template <bool kPaged>
__device__ __forceinline__ int unit_len(const Kv4Args &a, int b)
{
    if constexpr (kPaged) {
        int n = a.ctx_per_row ? 0 : a.ctx[b];
        if (a.ctx_per_row)
            for (int j = 0; j < a.next_n; ++j)
                n = max(n, a.ctx[(int64_t)b * a.next_n + j]);
        return min(max(n, 0), a.max_len);
    } else {
        const int64_t lo = min((int64_t)max(a.indptr[b], 0), a.num_slots);
        const int64_t hi = min((int64_t)max(a.indptr[b + 1], 0), a.num_slots);
        return (int)max((int64_t)0, hi - lo);
    }
}

// Tokens that row j of the unit sees.
template <bool kPaged>
__device__ __forceinline__ int row_end(const Kv4Args &a, int b, int j, int len)
{
    if constexpr (!kPaged)
        return len;
    const int n = a.ctx_per_row ? a.ctx[(int64_t)b * a.next_n + j]
                                : (int)max((int64_t)a.ctx[b] - a.next_n + j + 1, (int64_t)0);
    return min(max(n, 0), a.max_len);
}

// Every sequence counts a tile at least: its outputs are written.
template <bool kPaged>
__device__ __forceinline__ int64_t unit_tiles(const Kv4Args &a, int b)
{
    return a.uncut ? 1 : max(1, (int)(((int64_t)unit_len<kPaged>(a, b) + kTile - 1) / kTile));
}

// A share of the list: segments of units' tiles.  Sequences lie behind one
// another, each with its key heads and blocks of columns.
struct Share {
    int b, hc;       // sequence; key head x blocks of columns
    int tiles, len;  // of the sequence
    int t;           // next tile
    int left;        // tiles left
    int each, more;  // of all shares: size, how many have one more
};

// Sums over the block, for every thread: upto and including its own, and of all.
template <int kAllWarps>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *wsum, int64_t &all)
{
    const int lane = lane_id(), warp = threadIdx.x >> 5;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, v, o);
        v += lane >= o ? up : 0;
    }
    __syncthreads();
    if (lane == 31)
        wsum[warp] = v;
    __syncthreads();
    all = 0;
    #pragma unroll
    for (int i = 0; i < kAllWarps; ++i) {
        v += i < warp ? wsum[i] : 0;
        all += wsum[i];
    }
    return v;
}

// The share of this thread's group of kWarps warps (left: 0 where it has none);
// group i of a CTA takes share i * gridDim.x + blockIdx.x, so that few shares
// spread over the SMs.  limit: tiles that a list may have.
template <bool kPaged, int kGroups>
__device__ __forceinline__ void find_share(const Kv4Args &a, int heads, int64_t limit, Share &s)
{
    constexpr int kAll = kGroups * kThreads, kFew = 128;
    const int tid = threadIdx.x, lane = lane_id(), group = tid / kThreads;
    const int p = group * gridDim.x + blockIdx.x;
    s.left = s.each = s.more = 0;
    // tiles of all heads as one list, once it is known to be no longer than it may
    int shares = 0;
    const auto divide = [&](int64_t tiles) {
        if (tiles > limit) {
            if (blockIdx.x == 0 && tid == 0)
                atomicOr(a.status, kDevBadBounds);
            return false;
        }
        const uint32_t total = (uint32_t)(tiles * heads);
        shares = min(gridDim.x * kGroups, total);
        s.each = total / shares;
        s.more = total - s.each * shares;
        return true;
    };
    const auto begin = [&](int share) { return (int64_t)share * s.each + min(share, s.more); };
    int place;  // of the share's first tile among its sequence's
    if (a.B <= kFew) {
        // every warp by itself, four sequences a lane
        int n[kFew / 32];
        int64_t upto = 0;
        #pragma unroll
        for (int i = 0; i < kFew / 32; ++i) {
            const int b = kFew / 32 * lane + i;
            n[i] = b < a.B ? (int)unit_tiles<kPaged>(a, b) : 0;
            upto += n[i];
        }
        const int64_t mine = upto;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? up : 0;
        }
        if (!divide(__shfl_sync(0xffffffffu, upto, 31)) || p >= shares)
            return;
        int64_t at = begin(p) - (upto - mine) * heads;
        const uint32_t here = __ballot_sync(0xffffffffu, at >= 0 && at < mine * heads);
        int b = kFew / 32 * lane;
        #pragma unroll
        for (int i = 0; i + 1 < kFew / 32; ++i)
            if (at >= (int64_t)n[i] * heads && b == kFew / 32 * lane + i) {
                at -= (int64_t)n[i] * heads;
                ++b;
            }
        const int who = __ffs(here) - 1;
        s.b = __shfl_sync(0xffffffffu, b, who);
        place = __shfl_sync(0xffffffffu, (int)at, who);
    } else {
        __shared__ int64_t wsum[kGroups * kWarps];
        __shared__ int2 found[kGroups];
        int64_t total = 0, mine = 0, upto = 0, all;
        for (int b0 = 0; b0 < a.B; b0 += kAll) {
            mine = b0 + tid < a.B ? unit_tiles<kPaged>(a, b0 + tid) : 0;
            upto = total + block_scan<kGroups * kWarps>(mine, wsum, all);
            total += all;
        }
        if (!divide(total))
            return;
        const auto look = [&](int b) {
            const int64_t before = (upto - mine) * heads, after = before + mine * heads;
            #pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int64_t u = begin(i * gridDim.x + blockIdx.x);
                if (u >= before && u < after)
                    found[i] = make_int2(b, (int)(u - before));
            }
        };
        if (a.B <= kAll) {
            look(tid);
        } else {
            int64_t sum = 0;
            for (int b0 = 0; b0 < a.B; b0 += kAll) {
                mine = b0 + tid < a.B ? unit_tiles<kPaged>(a, b0 + tid) : 0;
                upto = sum + block_scan<kGroups * kWarps>(mine, wsum, all);
                sum += all;
                look(b0 + tid);
            }
        }
        __syncthreads();
        if (p >= shares)
            return;
        s.b = found[group].x;
        place = found[group].y;
    }
    s.left = s.each + (p < s.more);
    s.len = unit_len<kPaged>(a, s.b);
    s.tiles = (int)unit_tiles<kPaged>(a, s.b);
    s.hc = place / s.tiles;
    s.t = place - s.hc * s.tiles;
}

// The tiles that rows which are not cut list, though their shares count a unit each: of
// few rows four a lane, whose bounds are read beside the first look-ups and added up later.
struct Listed {
    static constexpr int kFew = 128, kEach = kFew / 32;
    int bound[kEach + 1];

    __device__ __forceinline__ void look(const Kv4Args &a)
    {
        if (a.B <= kFew)
            #pragma unroll
            for (int i = 0; i <= kEach; ++i)
                bound[i] = a.indptr[min(kEach * lane_id() + i, a.B)];
    }
    // Whether they are more than num_slots tokens in B rows have: one answer for all threads
    // of all CTAs.
    template <int kGroups>
    __device__ __forceinline__ bool too_many(const Kv4Args &a) const
    {
        const auto tiles = [&](int lo, int hi) {
            const int most = (int)a.num_slots;
            return max(1, (min(max(hi, 0), most) - min(max(lo, 0), most) + kTile - 1) / kTile);
        };
        const int64_t limit = a.num_slots / kTile + a.B;
        if (a.B <= kFew) {
            uint32_t n = 0;
            #pragma unroll
            for (int i = 0; i < kEach; ++i)
                n += kEach * lane_id() + i < a.B ? tiles(bound[i], bound[i + 1]) : 0;
            return __reduce_add_sync(0xffffffffu, n) > limit;
        }
        __shared__ int64_t wsum[kGroups * kWarps];
        int64_t n = 0, all;
        for (int b = threadIdx.x; b < a.B; b += kGroups * kThreads)
            n += tiles(a.indptr[b], a.indptr[b + 1]);
        block_scan<kGroups * kWarps>(n, wsum, all);
        return all > limit;
    }
};

// The share of a group of a team: of one unit's tiles, by its number among the team's.
// False where the rows list more than they may (there are no more rows than SMs).
template <bool kPaged, int kGroups>
__device__ __forceinline__ bool team_share(const Kv4Args &a, int heads, int64_t limit, Share &s)
{
    const int unit = blockIdx.x / a.team, groups = a.team * kGroups;
    const int nth = (blockIdx.x - unit * a.team) * kGroups + threadIdx.x / kThreads;
    s.b = unit / heads;
    s.hc = unit - s.b * heads;
    s.len = unit_len<kPaged>(a, s.b);
    s.tiles = max(1, (s.len + kTile - 1) / kTile);
    s.t = (int)((int64_t)s.tiles * nth / groups);
    s.left = (int)((int64_t)s.tiles * (nth + 1) / groups) - s.t;
    s.each = s.more = 0;
    if (kPaged || a.B == 1)
        return true;
    uint32_t tiles = 0;
    for (int b = lane_id(); b < a.B; b += 32)
        tiles += (uint32_t)unit_tiles<kPaged>(a, b);
    if (__reduce_add_sync(0xffffffffu, tiles) <= limit)
        return true;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        atomicOr(a.status, kDevBadBounds);
    s.left = 0;
    return false;
}

// A segment: tiles [t0, t1) of a unit.
struct Seg {
    int b, hc, len, t0, t1, tiles;
};

template <bool kPaged>
__device__ __forceinline__ bool next_seg(const Kv4Args &a, int heads, Share &s, Seg &g)
{
    if (s.left <= 0)
        return false;
    if (s.t == s.tiles) {
        s.t = 0;
        if (++s.hc == heads) {
            s.hc = 0;
            ++s.b;
            s.len = unit_len<kPaged>(a, s.b);
            s.tiles = (int)unit_tiles<kPaged>(a, s.b);
        }
    }
    const int n = min(s.left, s.tiles - s.t);
    g = {s.b, s.hc, s.len, s.t, s.t + n, s.tiles};
    s.t += n;
    s.left -= n;
    if (a.uncut)
        g.t1 = g.tiles = max(1, (s.len + kTile - 1) / kTile);
    return true;
}

// ------------------------------------------------------------------- a ring
//
// A warp's tokens on their way in: codes of the keys (and values), scales, and
// which tokens are there.  It is filled ahead of the walk, over the ends of
// segments; the walk that fills is a second one, in shared memory but for the
// segment at hand.  One place is always free: the one that was read last.
template <int kMode, bool kValues, int kStages>
struct Ring {
    static constexpr bool kPaged = kMode != kSlots;
    static constexpr int kCodes = (kValues ? 2 : 1) * kSubCodes;
    static constexpr int kScales = (kValues ? 2 : 1) * 4 * kSub;
    static constexpr int kStage = kCodes + kScales;
    // behind the stages: scales of the keys in 32 bits, of the values in 16, the second walk, and
    // which tokens are there
    static constexpr int kOffKeys = kStages * kStage;
    static constexpr int kOffValues = kOffKeys + 16 * kSub;
    static constexpr int kOffWalk = kOffValues + (kValues ? 8 * kSub : 0);
    static constexpr int kOffMasks = kOffWalk + 48;
    static constexpr int kBytes = (kOffMasks + 4 * kStages + 63) / 64 * 64;  // places lie at multiples of 64

    uint8_t *mem;
    int32_t ahead;         // the next step's slot, or its page
    int off;               // its tokens' place in the page
    const int32_t *from;   // the row's slots, or the sequence's pages
    int head, len;         // of the segment at hand
    int tok;               // slots, pages: this lane's next token; whole pages: the step's first
    int left;              // steps of the segment; negative: no more
    // whole pages: this lane's first piece of a page's keys and of its scales; the last
    // steps' pages outside the pool, a bit each
    uint32_t code_at, scale_at, bad;

    __device__ __forceinline__ uint8_t *stage(int i) const { return mem + i * kStage; }
    __device__ __forceinline__ float4 *key_scales() const
    {
        return reinterpret_cast<float4 *>(mem + kOffKeys);
    }
    __device__ __forceinline__ uint2 *value_scales() const
    {
        return reinterpret_cast<uint2 *>(mem + kOffValues);
    }
    __device__ __forceinline__ uint32_t *masks() const
    {
        return reinterpret_cast<uint32_t *>(mem + kOffMasks);
    }
    __device__ __forceinline__ Share *walk() const
    {
        return reinterpret_cast<Share *>(mem + kOffWalk);
    }
    __device__ __forceinline__ void look(const Kv4Args &a)
    {
        ahead = -1;
        if (tok < len) {
            if constexpr (kPaged) {
                const int block = page_of(a.pool.p, tok);
                ahead = from[block];
                off = tok - block * a.pool.p.page_size;
            } else {
                ahead = from[tok];
            }
        }
    }
    // The next segment of the second walk that has a step for this warp.
    __device__ __forceinline__ void advance(const Kv4Args &a, int heads, int blocks, int warp)
    {
        Share s = *walk();
        Seg g;
        do {
            left = -1;
            if (!next_seg<kPaged>(a, heads, s, g))
                break;
            const int tok0 = g.t0 * kTile + warp * kSub;
            len = (int)min((int64_t)g.t1 * kTile, (int64_t)g.len);
            left = tok0 < len ? (len - tok0 + kTile - 1) / kTile : 0;
            tok = tok0 + (kMode == kWholePages ? 0 : lane_id());
        } while (left == 0);
        __syncwarp();
        if (lane_id() == 0)
            *walk() = s;
        __syncwarp();
        if (left < 0)
            return;
        head = g.hc / blocks;
        off = 0;
        if constexpr (kMode == kWholePages) {
            const uint32_t token = (uint32_t)head * a.pool.p.page_size, lane = lane_id();
            code_at = token * kKv4Codes + 16 * lane;
            scale_at = (uint32_t)a.pool.scales + token * kKv4Groups +
                       (lane >> 3) * (uint32_t)a.pool.scale_side + 16 * (lane & 7);
        }
        if constexpr (kPaged)
            from = a.table + g.b * a.bt_stride;
        else
            from = a.slots + min((int64_t)max(a.indptr[g.b], 0), a.num_slots);
        look(a);
    }
    __device__ __forceinline__ void start(const Kv4Args &a, const Share &s, int heads, int blocks,
                                          int warp)
    {
        if (lane_id() == 0)
            *walk() = s;
        __syncwarp();
        left = 0;
        bad = 0;
        advance(a, heads, blocks, warp);
    }
    // One more step into place st, if there is one; a group of copies is committed in any case.
    __device__ __forceinline__ void fill(const Kv4Args &a, int heads, int blocks, int warp, int st)
    {
        if (left == 0)
            advance(a, heads, blocks, warp);
        bad <<= 1;
        if (left > 0) {
            --left;
            copy(a, st);
        }
        cp_async_commit();
    }
    // Which tokens of the step that is read next are there; rows: of the segment from its first
    // on.  (kStages - 1 steps were filled after it.)
    __device__ __forceinline__ uint32_t there(int st, int rows) const
    {
        if constexpr (kMode == kWholePages) {
            const uint32_t all = rows >= kSub ? 0xffffffffu : (1u << rows) - 1u;
            return bad >> (kStages - 1) & 1 ? 0u : all;
        } else {
            return masks()[st];
        }
    }
    __device__ __forceinline__ void copy(const Kv4Args &a, int st)
    {
        const int lane = lane_id();
        const uint32_t to = smem_u32(mem) + st * kStage;
        const uint32_t d = to + (lane >> 2) * kKv4Codes + 16 * ((lane & 3) ^ (lane >> 3));
        int page = ahead, o = off;
        if constexpr (kMode == kWholePages) {
            // 32 tokens side by side; those past the context lie in its last page too
            tok += kTile;
            look(a);
            if ((uint32_t)page < (uint32_t)a.pool.p.num_pages) {
                const uint8_t *base = a.pool.p.base + (uint64_t)(uint32_t)page * (uint32_t)a.pool.p.stride;
                const uint8_t *keys = base + (code_at + o * kKv4Codes);
                #pragma unroll
                for (int i = 0; i < 4; ++i)
                    cp_async16(d + i * 8 * kKv4Codes, keys + i * 8 * kKv4Codes);
                if constexpr (kValues) {
                    const uint8_t *vals = keys + (uint32_t)a.pool.side;
                    #pragma unroll
                    for (int i = 0; i < 4; ++i)
                        cp_async16(d + kSubCodes + i * 8 * kKv4Codes, vals + i * 8 * kKv4Codes);
                }
                if (lane < (kValues ? 16 : 8))
                    cp_async16(to + kCodes + 16 * lane, base + (scale_at + o * kKv4Groups));
            } else {
                bad |= 1;
                if (lane == 0)
                    atomicOr(a.status, kDevBadPage);
            }
        } else {
            bool good = tok < len;
            if constexpr (!kPaged) {
                if (page >= 0) {
                    const int slot = page;
                    page = page_of(a.pool.p, slot);
                    o = slot - page * a.pool.p.page_size;
                }
            }
            if (good && (page < 0 || page >= a.pool.p.num_pages)) {
                good = false;
                atomicOr(a.status, kDevBadPage);
            }
            tok += kTile;
            look(a);
            const uint32_t there = __ballot_sync(0xffffffffu, good);
            if (lane == 0)
                masks()[st] = there;
            const int64_t base = (uint64_t)(uint32_t)page * (uint32_t)a.pool.p.stride;
            const uint32_t token = (uint32_t)head * a.pool.p.page_size + o;
            const int64_t code = base + token * kKv4Codes;
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 8 * i + (lane >> 2);
                const uint8_t *keys = a.pool.p.base + __shfl_sync(0xffffffffu, code, row) + 16 * (lane & 3);
                if (there >> row & 1) {
                    cp_async16_alone(d + i * 8 * kKv4Codes, keys);
                    if constexpr (kValues)
                        cp_async16_alone(d + kSubCodes + i * 8 * kKv4Codes, keys + a.pool.side);
                }
            }
            if (good) {
                const uint8_t *sc = a.pool.p.base + base + (a.pool.scales + token * kKv4Groups);
                cp_async4_alone(to + kCodes + 4 * lane, sc);
                if constexpr (kValues)
                    cp_async4_alone(to + kCodes + 4 * (kSub + lane), sc + a.pool.scale_side);
            }
        }
    }
    // The scales of a step's keys in 32 bits, a lane a token (a warp's barrier follows).
    __device__ __forceinline__ void widen_key_scales(int st) const
    {
        float f[4];
        e8m0_to_float(reinterpret_cast<const uint32_t *>(stage(st) + kCodes)[lane_id()], f);
        key_scales()[lane_id()] = make_float4(f[0], f[1], f[2], f[3]);
    }
};

// ------------------------------------------------------------------- queries

// Query fragments of a block of columns, as f16 under a power of two for each
// column: eight columns' in registers, more in shared memory (16 columns on 16
// registers each of the sums' 64 and the step's own spill).
template <int NT>
struct Queries {
    static constexpr int kBytes = NT == 1 ? 0 : NT * 4 * 512;
    uint32_t r[NT == 1 ? 4 : 1][4];
    uint32_t at;  // shared memory: this lane's place

    __device__ __forceinline__ void put(int n, int i, const uint32_t (&v)[4])
    {
        if constexpr (NT == 1) {
            #pragma unroll
            for (int x = 0; x < 4; ++x)
                r[i][x] = v[x];
        } else {
            st_shared_v4(at + (4 * n + i) * 512, v[0], v[1], v[2], v[3]);
        }
    }
    __device__ __forceinline__ void get(int n, int i, uint32_t (&v)[4]) const
    {
        if constexpr (NT == 1) {
            #pragma unroll
            for (int x = 0; x < 4; ++x)
                v[x] = r[i][x];
        } else {
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(at + (4 * n + i) * 512));
        }
    }
};

// slc brings scores to units of log2 (columns 2 c, 2 c + 1 of each eight).
template <int NT>
__device__ __forceinline__ void load_queries(const Kv4Args &a, int b, int key_head, int cb,
                                             Queries<NT> &q, float (&slc)[NT][2])
{
    const int lane = lane_id(), g = lane >> 2, c = lane & 3;
    #pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int col = (cb * NT + n) * 8 + g, j = col / a.group;
        uint4 raw[4] = {};
        if (col < a.cols) {
            const uint16_t *src = a.q + ((int64_t)b * a.next_n + j) * a.ldq_row +
                                  (int64_t)(key_head * a.group + col - j * a.group) * a.ldq_head;
            #pragma unroll
            for (int i = 0; i < 4; ++i)
                raw[i] = *reinterpret_cast<const uint4 *>(src + 32 * i + 8 * c);
        }
        uint32_t top = 0;
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            #pragma unroll
            for (int e = 0; e < 4; ++e)
                top = max(top, max((w[e] << 16) & 0x7fffffffu, w[e] & 0x7fff0000u));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the largest to [2^14, 2^15), as far as the power's inverse times the scale is a
        // normal number (zero times the -inf of a masked score would be NaN; the queries that
        // stop short of it score nothing); infinities and NaN stay what they are
        const int e = (int)(top >> 23);
        const int most = max((int)(__float_as_uint(a.scale_log2) >> 23) - 1, 0);
        const int up = e == 0 || e == 255 ? 0 : min(141 - e, min(most, 126));
        const float f = __uint_as_float((uint32_t)(127 + up) << 23);
        const float back = __uint_as_float((uint32_t)(127 - up) << 23) * a.scale_log2;
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            uint32_t v[4];
            #pragma unroll
            for (int x = 0; x < 4; ++x)
                v[x] = as_u32(__floats2half2_rn(__uint_as_float(w[x] << 16) * f,
                                                __uint_as_float(w[x] & 0xffff0000u) * f));
            q.put(n, i, v);
        }
        #pragma unroll
        for (int i = 0; i < 2; ++i)
            slc[n][i] = __shfl_sync(0xffffffffu, back, (2 * c + i) * 4);
    }
}

// Scores of 32 tokens: s[m][n][0, 1] of token 16 m + g, [2, 3] of the one 8
// further, columns 2 c and 2 c + 1.
template <int NT>
__device__ __forceinline__ void score_tile(uint32_t codes, uint32_t scales, const Queries<NT> &q,
                                           float (&s)[2][NT][4])
{
    const int lane = lane_id(), g = lane >> 2, c = lane & 3;
    // (pieces of 16 bytes are turned by the row's number: places are multiples of 64)
    const uint32_t row = codes + g * kKv4Codes + 4 * c + ((g >> 1 & 3) << 4);
    float sc[2][2][4];  // of the two tiles' rows
    #pragma unroll
    for (int m = 0; m < 2; ++m)
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 v = lds128f(scales + 16 * g + 256 * m + 128 * h);
            sc[m][h][0] = v.x;
            sc[m][h][1] = v.y;
            sc[m][h][2] = v.z;
            sc[m][h][3] = v.w;
        }
    // A group's products are scaled, two columns at once, while the next one's run.
    float d[2][2][NT][4];
    #pragma unroll
    for (int i = 0; i < 5; ++i) {
        uint32_t a0[2][4], a1[2][4], b[NT][4];
        if (i < 4) {
            #pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint32_t ka[4], kb[4];
                e2m1_to_f16x2(lds32((row ^ (16 * i)) + 16 * m * kKv4Codes), ka);
                e2m1_to_f16x2(lds32((row ^ (16 * i)) + (16 * m + 8) * kKv4Codes), kb);
                #pragma unroll
                for (int x = 0; x < 2; ++x) {
                    a0[m][2 * x] = ka[x];
                    a0[m][2 * x + 1] = kb[x];
                    a1[m][2 * x] = ka[2 + x];
                    a1[m][2 * x + 1] = kb[2 + x];
                }
            }
            #pragma unroll
            for (int n = 0; n < NT; ++n) {
                q.get(n, i, b[n]);
                #pragma unroll
                for (int m = 0; m < 2; ++m)
                    mma16_first(d[i & 1][m][n], a0[m], b[n][0], b[n][1]);
            }
        }
        if (i > 0) {
            #pragma unroll
            for (int n = 0; n < NT; ++n)
                #pragma unroll
                for (int m = 0; m < 2; ++m)
                    #pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float f = sc[m][h][i - 1];
                        const float *v = d[~i & 1][m][n] + 2 * h;
                        const float2 t = i == 1
                            ? __fmul2_rn(make_float2(v[0], v[1]), make_float2(f, f))
                            : fma2(make_float2(v[0], v[1]), make_float2(f, f),
                                   make_float2(s[m][n][2 * h], s[m][n][2 * h + 1]));
                        s[m][n][2 * h] = t.x;
                        s[m][n][2 * h + 1] = t.y;
                    }
        }
        if (i < 4) {
            #pragma unroll
            for (int n = 0; n < NT; ++n)
                #pragma unroll
                for (int m = 0; m < 2; ++m)
                    mma16(d[i & 1][m][n], a1[m], b[n][2], b[n][3]);
        }
    }
}

// Scores of places where there is no token, or none that the column sees, are
// -inf.  tok0: the first token; ends of columns 2 c, 2 c + 1.
template <int NT>
__device__ __forceinline__ void mask_tile(float (&s)[2][NT][4], uint32_t there, int tok0,
                                          const int (&end)[NT][2])
{
    const int g = lane_id() >> 2;
    #pragma unroll
    for (int m = 0; m < 2; ++m)
        #pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int r = 16 * m + g + 8 * (x >> 1);
            const bool here = there >> r & 1;
            #pragma unroll
            for (int n = 0; n < NT; ++n)
                s[m][n][x] = here && tok0 + r < end[n][x & 1] ? s[m][n][x] : -INFINITY;
        }
}

// ----------------------------------------------------------------- attention

template <int NT>
struct Shape {
    static constexpr int kCols = 8 * NT;
    static constexpr int kStages = 2;  // (three: no faster, and less of L1)
    // Groups of kWarps warps with shares of their own: an SM has one CTA of as many as
    // registers and shared memory hold.
    static constexpr int kGroups = NT == 1 ? 4 : 3;
    static constexpr int kPart = kCols * (kKv4Dim + 2);  // floats of a partial result
    static constexpr int kRow = kKv4Dim + 4;  // of a column in a team's shared memory: a quad's columns
                                              // fall into different banks
    template <int kMode>
    static constexpr int smem()
    {
        return kGroups * (kWarps * Ring<kMode, true, kStages>::kBytes + 2 * Queries<NT>::kBytes);
    }
};

// A warp's sums: O in absolute units, of element tiles x columns, maxima, sums of
// the weights.
template <int NT>
struct Sums {
    float o[8][NT][4], m[NT][2], l[NT][2];
};

// Sums go from one warp to another through the first one's free place, a block of
// eight columns at a time, with a barrier of the two before and after it is read.
template <int NT>
__device__ __forceinline__ void give_sums(const Sums<NT> &s, uint8_t *place, int barrier)
{
    const int lane = lane_id();
    float4 *to = reinterpret_cast<float4 *>(place);
    #pragma unroll
    for (int n = 0; n < NT; ++n) {
        #pragma unroll
        for (int x = 0; x < 8; ++x)
            to[32 * x + lane] = make_float4(s.o[x][n][0], s.o[x][n][1], s.o[x][n][2], s.o[x][n][3]);
        if (lane < 4)  // the columns' maxima and sums are the quads' alike
            to[256 + lane] = make_float4(s.m[n][0], s.m[n][1], s.l[n][0], s.l[n][1]);
        named_bar_sync(barrier, 64);
        named_bar_sync(barrier, 64);  // it was read
    }
}

template <int NT, typename Place>
__device__ __forceinline__ void take_sums(Sums<NT> &s, Place place, int warp, int barrier)
{
    const int lane = lane_id();
    #pragma unroll
    for (int n = 0; n < NT; ++n) {
        named_bar_sync(barrier, 64);
        const float4 *from = reinterpret_cast<const float4 *>(place(warp));
        const float4 st = from[256 + (lane & 3)];
        const float m[2] = {st.x, st.y}, l[2] = {st.z, st.w};
        float mine[2], theirs[2];
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float top = fmaxf(s.m[n][i], m[i]);
            mine[i] = ex2(s.m[n][i] - top);
            theirs[i] = ex2(m[i] - top);
            s.m[n][i] = top;
            s.l[n][i] = s.l[n][i] * mine[i] + l[i] * theirs[i];
        }
        #pragma unroll
        for (int x = 0; x < 8; ++x) {
            const float4 v = from[32 * x + lane];
            const float o[4] = {v.x, v.y, v.z, v.w};
            #pragma unroll
            for (int e = 0; e < 4; ++e)
                s.o[x][n][e] = s.o[x][n][e] * mine[e & 1] + o[e] * theirs[e & 1];
        }
        named_bar_sync(barrier, 64);
    }
}

// A team's sums, joined by its CTAs, a column a warp; idle: this thread's group had no tile.
template <int NT, int kRingBytes>
__device__ __forceinline__ void join_team(const Kv4Args &a, uint8_t *smem, int b, int hc, bool idle)
{
    namespace cg = cooperative_groups;
    using S = Shape<NT>;
    constexpr int kCols = S::kCols, kGroups = S::kGroups, kAtOnce = 8;
    const int lane = lane_id(), warp = threadIdx.x >> 5, group = warp / kWarps;
    float *all = reinterpret_cast<float *>(smem);
    constexpr int kStep = kWarps * kRingBytes / 4;  // floats between groups
    constexpr int kStat = kCols * S::kRow;
    if (idle && warp % kWarps == 0 && lane < kCols) {
        all[group * kStep + kStat + lane] = -FLT_MAX;
        all[group * kStep + kStat + kCols + lane] = 0.0f;
    }
    cg::cluster_group team = cg::this_cluster();
    team.sync();
    const int head = hc / a.blocks, cb = hc - head * a.blocks;
    const int rank = (int)team.block_rank(), groups = a.team * kGroups;
    for (int col = rank + a.team * warp; col < min(kCols, a.cols - cb * kCols);
         col += a.team * kGroups * kWarps) {
        float top = -FLT_MAX, sum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int i0 = 0; i0 < groups; i0 += kAtOnce) {
            float m[kAtOnce], l[kAtOnce];
            float4 v[kAtOnce];
            #pragma unroll
            for (int x = 0; x < kAtOnce; ++x) {
                const int i = i0 + x;
                m[x] = -FLT_MAX;
                l[x] = 0.0f;
                v[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (i < groups) {
                    const float *f = team.map_shared_rank(all, i / kGroups) + i % kGroups * kStep;
                    m[x] = f[kStat + col];
                    l[x] = f[kStat + kCols + col];
                    v[x] = *reinterpret_cast<const float4 *>(f + col * S::kRow + 4 * lane);
                }
            }
            #pragma unroll
            for (int x = 0; x < kAtOnce; ++x) {
                if (l[x] == 0.0f)  // no sums were written
                    continue;
                const float up = fmaxf(top, m[x]), mine = ex2(top - up), w = ex2(m[x] - up);
                top = up;
                sum = sum * mine + l[x] * w;
                acc.x = acc.x * mine + v[x].x * w;
                acc.y = acc.y * mine + v[x].y * w;
                acc.z = acc.z * mine + v[x].z * w;
                acc.w = acc.w * mine + v[x].w * w;
            }
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const int at = cb * kCols + col, j = at / a.group, h = head * a.group + at - j * a.group;
        const int64_t row = (int64_t)b * a.next_n + j;
        *reinterpret_cast<uint2 *>(a.out + row * a.ldo_row + h * a.ldo_head + 4 * lane) =
            make_uint2(as_u32(__floats2bfloat162_rn(acc.x * inv, acc.y * inv)),
                       as_u32(__floats2bfloat162_rn(acc.z * inv, acc.w * inv)));
        if (a.lse && lane == 0)
            a.lse[row * a.ld_lse + h] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
    team.sync();  // the sums are read
}

// kListed: rows by slots that are not cut, whose tiles are counted against the slots' (an
// instance of its own: the count costs calls that go without it 0.2 us).
template <int kMode, int NT, bool kTeam, bool kListed>
__global__ void __launch_bounds__(Shape<NT>::kGroups * kThreads, 1)
    kv4_attention_kernel(const __grid_constant__ Kv4Args a)
{
    using S = Shape<NT>;
    using R = Ring<kMode, true, S::kStages>;
    constexpr bool kPaged = kMode != kSlots;
    constexpr int kStages = S::kStages, kCols = S::kCols, kGroups = S::kGroups;
    static_assert(R::kStage >= 257 * 16 && R::kStage % 64 == 0, "a place takes sums");
    static_assert(sizeof(Share) <= 48, "the second walk's place");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ volatile int places[kGroups * kWarps];  // the warps' free places, where they give sums
    const int lane = lane_id(), g = lane >> 2, c = lane & 3;
    const int all_warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int group = all_warp / kWarps, warp = all_warp % kWarps;  // of the group
    const int p = group * gridDim.x + blockIdx.x;                   // the group's share
    pdl_wait();
    pdl_launch_dependents();
    const int heads = a.pool.heads * a.blocks;
    const int64_t limit = kPaged || a.uncut ? INT64_MAX / INT_MAX : a.num_slots / kTile + a.B;
    const bool cuts = !kTeam && !a.uncut;
    if (warp == 0 && lane == 0 && cuts && !a.by_unit)
        a.ws_cut[p] = make_int4(0, 0, 0, 0);
    Listed listed;
    if constexpr (kListed)
        listed.look(a);
    Share share;
    bool good = true;
    if constexpr (kTeam)
        good = team_share<kPaged, kGroups>(a, heads, limit, share);
    else
        find_share<kPaged, kGroups>(a, heads, limit, share);
    const int unit_b = share.b, unit_hc = share.hc;  // a team's
    // a list that is left alone (shares of nothing) has nothing to join
    if (warp == 0 && lane == 0 && a.by_unit && cuts && share.each == 0 && p < a.B * heads)
        a.ws_cut[p] = make_int4(0, 0, 0, 0);
    R ring;
    ring.mem = smem + all_warp * R::kBytes;
    ring.start(a, share, heads, a.blocks, warp);
    #pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        ring.fill(a, heads, a.blocks, warp, i);
    if constexpr (kListed)
        if (listed.too_many<kGroups>(a)) {  // (the first copies are on their way)
            if (blockIdx.x == 0 && threadIdx.x == 0)
                atomicOr(a.status, kDevBadBounds);
            share.left = 0;
        }
    int st = 0;            // the next place to read
    int spare = kStages - 1;  // the free one
    Seg seg;
    const bool idle = share.left == 0;
    for (int nth = 0; next_seg<kPaged>(a, heads, share, seg); ++nth) {
        const int head = seg.hc / a.blocks, cb = seg.hc - head * a.blocks;
        const int tok0 = seg.t0 * kTile + warp * kSub;
        const int upto = (int)min((int64_t)seg.t1 * kTile, (int64_t)seg.len);
        const int steps = tok0 < upto ? (upto - tok0 + kTile - 1) / kTile : 0;
        // A group's warps write the same fragments.  They are a segment apart at most: by turns
        // into two places.
        Queries<NT> qf;
        qf.at = smem_u32(smem) + kGroups * kWarps * R::kBytes +
                (2 * group + (nth & 1)) * Queries<NT>::kBytes + 16 * lane;
        float slc[NT][2];
        load_queries<NT>(a, seg.b, head, cb, qf, slc);
        __syncwarp();
        int end[NT][2], least = INT_MAX;
        #pragma unroll
        for (int n = 0; n < NT; ++n)
            #pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = cb * kCols + n * 8 + 2 * c + i;
                end[n][i] = col < a.cols ? row_end<kPaged>(a, seg.b, col / a.group, seg.len) : 0;
                if (col < a.cols)
                    least = min(least, end[n][i]);
            }
        least = __reduce_min_sync(0xffffffffu, least);

        Sums<NT> sum;
        // element tiles: rows 32 (t / 2) + 4 g + 2 (t % 2) and the next
        auto &o = sum.o;
        auto &m = sum.m;
        auto &l = sum.l;
        #pragma unroll
        for (int n = 0; n < NT; ++n) {
            #pragma unroll
            for (int x = 0; x < 8; ++x)
                #pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[x][n][i] = 0.0f;
            #pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[n][i] = -FLT_MAX;
                l[n][i] = 0.0f;
            }
        }
        uint32_t top_e = 0;  // the largest exponents, a byte a group
        #pragma unroll 1
        for (int k = 0; k < steps; ++k) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            ring.fill(a, heads, a.blocks, warp, spare);
            ring.widen_key_scales(st);
            const uint8_t *mem = ring.stage(st);
            const uint32_t *scales = reinterpret_cast<const uint32_t *>(mem + R::kCodes) + kSub;
            const int tok = tok0 + k * kTile;
            const uint32_t there = ring.there(st, upto - tok);
            spare = st;
            st = st + 1 == kStages ? 0 : st + 1;

            // ---- exponents of the values: a lane a token, two groups a word (0 and 2, 1 and 3)
            const bool here = there >> lane & 1;
            const uint32_t word = here ? scales[lane] : top_e;
            uint32_t under[2];  // the tops less them, in halves
            const auto in_range = [&](uint32_t w) {
                // (one over the top is negative, which shows in its upper bits)
                under[0] = (top_e & 0x00ff00ffu) - (w & 0x00ff00ffu);
                under[1] = (top_e >> 8 & 0x00ff00ffu) - (w >> 8 & 0x00ff00ffu);
                static_assert(kScaleRange == 15, "four bits");
                return ((under[0] | under[1]) & 0xfff0fff0u) == 0;
            };
            bool fast = __all_sync(0xffffffffu, in_range(word));
            if (!fast) {
                // raise the tops over this step's (one more, so that the next need not), NaN apart
                uint32_t t = here ? word & ~__vcmpeq4(word, 0xffffffffu) : 0u;
                #pragma unroll
                for (int x = 16; x > 0; x >>= 1)
                    t = __vmaxu4(t, __shfl_xor_sync(0xffffffffu, t, x));
                uint32_t next = 0;
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int was = top_e >> (8 * i) & 255, now = t >> (8 * i) & 255;
                    const int e = now > was ? min(now + 1, 254) : was;
                    next |= (uint32_t)e << (8 * i);
                    const float f = pow2i(was - e);
                    #pragma unroll
                    for (int n = 0; n < NT; ++n)
                        #pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            o[2 * i][n][x] *= f;
                            o[2 * i + 1][n][x] *= f;
                        }
                }
                top_e = next;
                fast = __all_sync(0xffffffffu, in_range(here ? word : top_e));
            }
            {
                // the token's scales as f16, 2^(e - top + 1) by their exponent bits; two lanes
                // change halves, so that pairs of tokens lie together
                const uint32_t f0 = 0x00010001u * ((15 + kScaleUp) << 10) - under[0] * 1024u;
                const uint32_t f1 = 0x00010001u * ((15 + kScaleUp) << 10) - under[1] * 1024u;
                const bool odd = lane & 1;
                const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? f0 : f1, 1);
                const uint32_t x = odd ? got : f0, y = odd ? f1 : got;
                ring.value_scales()[lane] = make_uint2(__byte_perm(x, y, 0x5410), __byte_perm(x, y, 0x7632));
            }
            __syncwarp();

            float s[2][NT][4];
            score_tile<NT>(smem_u32(mem), smem_u32(ring.key_scales()), qf, s);
            if (there != 0xffffffffu || tok + kSub > least)
                mask_tile<NT>(s, there, tok, end);

            // ---- the running maximum
            bool over = false;
            float mx[NT][2];
            #pragma unroll
            for (int n = 0; n < NT; ++n)
                #pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mx[n][i] = fmaxf(fmaxf(s[0][n][i], s[0][n][i + 2]),
                                     fmaxf(s[1][n][i], s[1][n][i + 2])) * slc[n][i];
                    over |= mx[n][i] > m[n][i] + kLazy;
                }
            if (__any_sync(0xffffffffu, over)) {
                #pragma unroll
                for (int n = 0; n < NT; ++n)
                    #pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float t = mx[n][i];
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                        const float nm = fmaxf(m[n][i], t);
                        const float al = nm == m[n][i] ? 1.0f : ex2(m[n][i] - nm);
                        m[n][i] = nm;
                        l[n][i] *= al;
                        #pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            o[x][n][i] *= al;
                            o[x][n][i + 2] *= al;
                        }
                    }
            }
            // ---- weights
            #pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 f = make_float2(slc[n][0], slc[n][1]);
                const float2 z = make_float2((float)kBias - m[n][0], (float)kBias - m[n][1]);
                float2 all = make_float2(l[n][0], l[n][1]);
                #pragma unroll
                for (int h = 0; h < 2; ++h)
                    #pragma unroll
                    for (int x = 0; x < 4; x += 2) {
                        float2 t = fma2(make_float2(s[h][n][x], s[h][n][x + 1]), f, z);
                        t = make_float2(ex2(t.x), ex2(t.y));
                        s[h][n][x] = t.x;
                        s[h][n][x + 1] = t.y;
                        all = __fadd2_rn(all, t);
                    }
                l[n][0] = all.x;
                l[n][1] = all.y;
            }

            // element pairs of groups 2 y and 2 y + 1 of four tokens, widened: rows of the
            // products' left side, two tiles a group
            const uint32_t val = smem_u32(mem) + kSubCodes + 2 * c * kKv4Codes + 2 * g + (c << 4);
            const auto widen = [&](int h, int y, uint32_t (&w)[4][4]) {
                uint32_t r[4];
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = (16 * h + (i & 1) + 8 * (i >> 1)) * kKv4Codes;
                    r[i] = __byte_perm(lds16((val ^ (32 * y)) + at), lds16((val ^ (32 * y + 16)) + at), 0x5410);
                }
                #pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t x0 = r[2 * i], x1 = r[2 * i + 1];
                    uint32_t f[4];
                    e2m1_to_f16x2((x0 & 0x0f0f0f0fu) | (x1 << 4 & 0xf0f0f0f0u), f);
                    #pragma unroll
                    for (int t = 0; t < 4; ++t)
                        w[t][2 * i] = f[t];
                    e2m1_to_f16x2((x0 >> 4 & 0x0f0f0f0fu) | (x1 & 0xf0f0f0f0u), f);
                    #pragma unroll
                    for (int t = 0; t < 4; ++t)
                        w[t][2 * i + 1] = f[t];
                }
            };
            if (fast) {
                #pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[NT][2];
                    #pragma unroll
                    for (int n = 0; n < NT; ++n)
                        #pragma unroll
                        for (int i = 0; i < 2; ++i)
                            p[n][i] = turn8(as_u32(__floats2half2_rn(s[h][n][2 * i], s[h][n][2 * i + 1])));
                    // groups 0, 2, 1, 3 of tokens 2 c, 2 c + 1 and of those 8 further
                    const uint4 e0 = *reinterpret_cast<const uint4 *>(ring.value_scales() + 16 * h + 2 * c);
                    const uint4 e1 = *reinterpret_cast<const uint4 *>(ring.value_scales() + 16 * h + 2 * c + 8);
                    const uint32_t fa[4] = {e0.x, e0.z, e0.y, e0.w}, fb[4] = {e1.x, e1.z, e1.y, e1.w};
                    #pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        uint32_t v[4][4];
                        widen(h, y, v);
                        #pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            #pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const uint32_t b0 = as_u32(__hmul2(as_h2(p[n][0]), as_h2(fa[2 * y + i])));
                                const uint32_t b1 = as_u32(__hmul2(as_h2(p[n][1]), as_h2(fb[2 * y + i])));
                                mma16(o[4 * y + 2 * i][n], v[2 * i], b0, b1);
                                mma16(o[4 * y + 2 * i + 1][n], v[2 * i + 1], b0, b1);
                            }
                        }
                    }
                }
            } else {
                // weights and scales in bf16; a column that does not see a token has no part
                // in a scale that is not finite
                #pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[NT][2], seen[NT] = {};
                    #pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        #pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float x = h ? s[1][n][2 * i] : s[0][n][2 * i];
                            const float y = h ? s[1][n][2 * i + 1] : s[0][n][2 * i + 1];
                            p[n][i] = turn8(as_u32(__floats2bfloat162_rn(x, y)));
                        }
                        const int col = cb * kCols + n * 8 + g;
                        const int last = col < a.cols ? row_end<kPaged>(a, seg.b, col / a.group, seg.len) : 0;
                        #pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int r = 16 * h + 2 * c + (x & 1) + 8 * (x >> 1);
                            seen[n] |= (uint32_t)((there >> r & 1) && tok + r < last) << x;
                        }
                    }
                    #pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        uint32_t v[4][4];
                        widen(h, y, v);
                        #pragma unroll
                        for (int t = 0; t < 4; ++t)
                            #pragma unroll
                            for (int x = 0; x < 4; ++x)
                                v[t][x] = to_bf16x2(v[t][x]);
                        #pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int grp = 2 * y + i;
                            float f[4];
                            #pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const int r = 16 * h + 2 * c + (x & 1) + 8 * (x >> 1);
                                const int e = scales[r] >> (8 * grp) & 255;
                                const int d = e - (int)(top_e >> (8 * grp) & 255) + kScaleUp;
                                f[x] = e == 255 ? NAN : pow2i(d);
                            }
                            #pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                uint32_t b[2];
                                #pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    const float2 pf = __bfloat1622float2(as_b2(p[n][x]));
                                    b[x] = as_u32(__floats2bfloat162_rn(
                                        seen[n] >> (2 * x) & 1 ? pf.x * f[2 * x] : 0.0f,
                                        seen[n] >> (2 * x + 1) & 1 ? pf.y * f[2 * x + 1] : 0.0f));
                                }
                                mma16_bf(o[4 * y + 2 * i][n], v[2 * i], b[0], b[1]);
                                mma16_bf(o[4 * y + 2 * i + 1][n], v[2 * i + 1], b[0], b[1]);
                            }
                        }
                    }
                }
            }
        }
        // ---- the warps' sums, in absolute units, from 1 to 0 and 3 to 2, then 2 to 0
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            // 2^(e - 127) less what the weights were raised by, by its bits: it may lie under the
            // least normal number, where the instruction for powers gives zero
            constexpr int kRaised = kScaleUp + kBias;
            const int e = top_e >> (8 * i) & 255;
            const float f = __uint_as_float(e > kRaised ? (uint32_t)(e - kRaised) << 23
                                                        : 0x400000u >> (kRaised - e));
            #pragma unroll
            for (int n = 0; n < NT; ++n)
                #pragma unroll
                for (int x = 0; x < 4; ++x) {
                    o[2 * i][n][x] *= f;
                    o[2 * i + 1][n][x] *= f;
                }
        }
        #pragma unroll
        for (int n = 0; n < NT; ++n)
            #pragma unroll
            for (int i = 0; i < 2; ++i) {
                float t = l[n][i];
                t += __shfl_xor_sync(0xffffffffu, t, 4);
                t += __shfl_xor_sync(0xffffffffu, t, 8);
                t += __shfl_xor_sync(0xffffffffu, t, 16);
                l[n][i] = t * pow2i(-kBias);
            }
        __syncwarp();  // the last step's place is read, and free
        if (warp > 0 && lane == 0)
            places[all_warp] = spare;
        if (warp & 1) {
            give_sums<NT>(sum, ring.stage(spare), 3 * group + 1 + (warp >> 1));
            continue;
        }
        // (a place's number is written before the barrier that tells of it)
        const auto place = [&](int w) {
            return smem + w * R::kBytes + places[w] * R::kStage;
        };
        take_sums<NT>(sum, place, all_warp + 1, 3 * group + 1 + (warp >> 1));
        if (warp == 2) {
            give_sums<NT>(sum, ring.stage(spare), 3 * group + 3);
            continue;
        }
        take_sums<NT>(sum, place, all_warp + 2, 3 * group + 3);

        // ---- warp 0 has the segment's
        if constexpr (kTeam) {
            // (the group's rings are read, and nothing is in flight)
            float *mine = reinterpret_cast<float *>(smem + group * kWarps * R::kBytes);
            #pragma unroll
            for (int n = 0; n < NT; ++n)
                #pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int col = n * 8 + 2 * c + i;
                    #pragma unroll
                    for (int y = 0; y < 4; ++y)
                        *reinterpret_cast<float4 *>(mine + col * S::kRow + 32 * y + 4 * g) =
                            make_float4(o[2 * y][n][i], o[2 * y][n][i + 2], o[2 * y + 1][n][i],
                                        o[2 * y + 1][n][i + 2]);
                    if (g == 0) {
                        mine[kCols * S::kRow + col] = m[n][i];
                        mine[kCols * (S::kRow + 1) + col] = l[n][i];
                    }
                }
            continue;
        }
        const bool part = seg.t0 > 0 || seg.t1 < seg.tiles;
        float *to = a.ws_part + (int64_t)(2 * p + (nth > 0)) * S::kPart;
        if ((part || a.by_unit) && cuts && seg.t0 == 0 && lane == 0) {
            // the shares that hold the rest: `more - p - 1` longer ones first
            const int longer = max(0, share.more - p - 1), rest = seg.tiles - seg.t1;
            const int in = (int)min((int64_t)rest, (int64_t)longer * (share.each + 1));
            a.ws_cut[a.by_unit ? seg.b * heads + seg.hc : p] = make_int4(
                seg.b, seg.hc, 1 + (in + share.each) / (share.each + 1) +
                                   (rest - in + share.each - 1) / share.each, 2 * p + (nth > 0));
        }
        #pragma unroll
        for (int n = 0; n < NT; ++n)
            #pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = n * 8 + 2 * c + i, at = cb * kCols + col;
                if (at >= a.cols)
                    continue;
                const float all = l[n][i];
                if (part) {
                    #pragma unroll
                    for (int y = 0; y < 4; ++y)
                        *reinterpret_cast<float4 *>(to + col * kKv4Dim + 32 * y + 4 * g) =
                            make_float4(o[2 * y][n][i], o[2 * y][n][i + 2], o[2 * y + 1][n][i],
                                        o[2 * y + 1][n][i + 2]);
                    if (g == 0) {
                        to[kCols * kKv4Dim + col] = m[n][i];
                        to[kCols * kKv4Dim + kCols + col] = all;
                    }
                } else {
                    const int j = at / a.group, h = head * a.group + at - j * a.group;
                    const int64_t row = (int64_t)seg.b * a.next_n + j;
                    const float inv = all == 0.0f ? 0.0f : 1.0f / all;
                    uint16_t *out = a.out + row * a.ldo_row + h * a.ldo_head + 4 * g;
                    #pragma unroll
                    for (int y = 0; y < 4; ++y)
                        *reinterpret_cast<uint2 *>(out + 32 * y) = make_uint2(
                            as_u32(__floats2bfloat162_rn(o[2 * y][n][i] * inv, o[2 * y][n][i + 2] * inv)),
                            as_u32(__floats2bfloat162_rn(o[2 * y + 1][n][i] * inv,
                                                         o[2 * y + 1][n][i + 2] * inv)));
                    if (a.lse && g == 0)
                        a.lse[row * a.ld_lse + h] =
                            all == 0.0f ? -INFINITY : (m[n][i] + log2f(all)) * kLn2;
                }
            }
    }
    cp_async_wait<0>();
    if constexpr (kTeam)
        if (good)  // (one answer for all CTAs)
            join_team<NT, R::kBytes>(a, smem, unit_b, unit_hc, idle);
}

// Joins the pieces of a unit that several shares hold, blockIdx.x its entry.  A
// block's warps take a column each, or all of them one column and every eighth
// piece; four pieces at once, under a running maximum.
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const Kv4Args a, int kCols, int together)
{
    constexpr int kTeams = kJoinThreads / 32, kAtOnce = 4;
    __shared__ float4 meet[kTeams][32];
    __shared__ float2 meet_stat[kTeams];
    const int warp = threadIdx.x >> 5, lane = lane_id();
    const int team = together ? warp : 0, teams = together ? kTeams : 1;
    const int col = together ? blockIdx.y : blockIdx.y * kTeams + warp;
    pdl_wait();
    pdl_launch_dependents();
    const int4 cut = a.ws_cut[blockIdx.x];
    const int pieces = cut.z;
    if (pieces < 2)
        return;
    const int head = cut.y / a.blocks, cb = cut.y - head * a.blocks;
    const int at = cb * kCols + col;
    if (col >= kCols || at >= a.cols)
        return;
    const int64_t step = 2 * (int64_t)kCols * (kKv4Dim + 2);
    const float *rest = a.ws_part + (cut.w >> 1) * step;
    const float *first = rest + (cut.w & 1) * (step / 2);
    float top = -FLT_MAX, sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const auto add = [&](float m, float l, float4 v) {
        const float up = fmaxf(top, m), mine = ex2(top - up), w = ex2(m - up);
        top = up;
        sum = sum * mine + l * w;
        acc.x = acc.x * mine + v.x * w;
        acc.y = acc.y * mine + v.y * w;
        acc.z = acc.z * mine + v.z * w;
        acc.w = acc.w * mine + v.w * w;
    };
    for (int i0 = team; i0 < pieces; i0 += kAtOnce * teams) {
        float m[kAtOnce], l[kAtOnce];
        float4 v[kAtOnce];
        #pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
            const int i = i0 + x * teams;
            const float *f = (i == 0 ? first : rest + i * step) + col * kKv4Dim;
            m[x] = -FLT_MAX;
            l[x] = 0.0f;
            v[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i < pieces) {
                m[x] = f[kCols * kKv4Dim - col * (kKv4Dim - 1)];
                l[x] = f[kCols * (kKv4Dim + 1) - col * (kKv4Dim - 1)];
                v[x] = *reinterpret_cast<const float4 *>(f + 4 * lane);
            }
        }
        #pragma unroll
        for (int x = 0; x < kAtOnce; ++x)
            add(m[x], l[x], v[x]);
    }
    if (together) {
        meet[team][lane] = acc;
        if (lane == 0)
            meet_stat[team] = make_float2(top, sum);
        __syncthreads();
        if (team > 0)
            return;
        #pragma unroll
        for (int i = 1; i < kTeams; ++i)
            add(meet_stat[i].x, meet_stat[i].y, meet[i][lane]);
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int j = at / a.group, h = head * a.group + at - j * a.group;
    const int64_t row = (int64_t)cut.x * a.next_n + j;
    *reinterpret_cast<uint2 *>(a.out + row * a.ldo_row + h * a.ldo_head + 4 * lane) =
        make_uint2(as_u32(__floats2bfloat162_rn(acc.x * inv, acc.y * inv)),
                   as_u32(__floats2bfloat162_rn(acc.z * inv, acc.w * inv)));
    if (a.lse && lane == 0)
        a.lse[row * a.ld_lse + h] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// ------------------------------------------------------------ tokens' weights
//
// The scores once more, without values: exp(s - lse) summed over the columns.
// Half the cache's bytes, and 8 of the weights.  Where there are more columns than a
// block, a segment is walked for each and the same lane adds to what it wrote.
template <int NT>
struct WeightShape {
    static constexpr int kStages = 4;
    static constexpr int kGroups = NT == 4 ? 3 : 4;
    template <int kMode>
    static constexpr int smem()
    {
        return kGroups * kWarps * (Ring<kMode, false, kStages>::kBytes + Queries<NT>::kBytes);
    }
};

template <int kMode, int NT>
__global__ void __launch_bounds__(WeightShape<NT>::kGroups * kThreads, 1)
    kv4_weights_kernel(const __grid_constant__ Kv4Args a)
{
    constexpr int kStages = WeightShape<NT>::kStages, kGroups = WeightShape<NT>::kGroups;
    constexpr int kCols = 8 * NT;
    using R = Ring<kMode, false, kStages>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = lane_id(), c = lane & 3;
    const int all_warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), warp = all_warp % kWarps;
    pdl_wait();
    pdl_launch_dependents();
    const int heads = a.pool.heads;
    Share share;
    find_share<true, kGroups>(a, heads, INT64_MAX / INT_MAX, share);
    R ring;
    ring.mem = smem + all_warp * R::kBytes;
    Queries<NT> qf;
    qf.at = smem_u32(smem) + kGroups * kWarps * R::kBytes + all_warp * Queries<NT>::kBytes + 16 * lane;
    Seg seg;
    while (next_seg<true>(a, heads, share, seg)) {
        const int head = seg.hc;
        const int tok0 = seg.t0 * kTile + warp * kSub;
        const int upto = (int)min((int64_t)seg.t1 * kTile, (int64_t)seg.len);
        const int steps = tok0 < upto ? (upto - tok0 + kTile - 1) / kTile : 0;
        const float *mass = a.mass ? a.mass + seg.b * a.ld_batch + head * a.ld_head : nullptr;
        float *out = a.mass_out + seg.b * a.ldo_batch + head * a.ldo_mass_head;
        // a walk of this segment alone
        Share one = {seg.b, seg.hc, seg.tiles, seg.len, seg.t0, seg.t1 - seg.t0, 0, 0};
        #pragma unroll 1
        for (int cb = 0; cb < a.blocks; ++cb) {
            ring.start(a, one, heads, 1, warp);
            #pragma unroll
            for (int i = 0; i < kStages - 1; ++i)
                ring.fill(a, heads, 1, warp, i);
            float slc[NT][2], z[NT][2];
            load_queries<NT>(a, seg.b, head, cb, qf, slc);
            __syncwarp();
            int end[NT][2], least = INT_MAX;
            #pragma unroll
            for (int n = 0; n < NT; ++n)
                #pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int col = cb * kCols + n * 8 + 2 * c + i, j = col / a.group;
                    end[n][i] = 0;
                    z[n][i] = -INFINITY;  // a column that is not there weighs nothing
                    if (col < a.cols) {
                        end[n][i] = row_end<true>(a, seg.b, j, seg.len);
                        const float v = a.lse_in[((int64_t)seg.b * a.next_n + j) * a.ld_lse_in +
                                                 (head * a.group + col - j * a.group) * a.ld_lse_head];
                        z[n][i] = v == -INFINITY ? 0.0f : -v * kLog2e;
                        least = min(least, end[n][i]);
                    }
                }
            least = __reduce_min_sync(0xffffffffu, least);
            // this lane's token of a step's sums: 16 (c / 2) + 8 (c % 2) + g; what it adds to
            // comes a step ahead
            int mine = tok0 + 16 * (c >> 1) + 8 * (c & 1) + (lane >> 2);
            const float *base = cb > 0 ? out : mass;
            float next = base && mine < upto ? base[mine] : 0.0f;
            int st = 0;
            #pragma unroll 1
            for (int k = 0; k < steps; ++k, mine += kTile) {
                const float before = next;
                next = base && mine < upto - kTile ? base[mine + kTile] : 0.0f;
                cp_async_wait<kStages - 2>();
                __syncwarp();
                ring.fill(a, heads, 1, warp, st == 0 ? kStages - 1 : st - 1);
                ring.widen_key_scales(st);
                const int tok = tok0 + k * kTile;
                const uint8_t *mem = ring.stage(st);
                const uint32_t there = ring.there(st, upto - tok);
                st = st + 1 == kStages ? 0 : st + 1;
                __syncwarp();
                float s[2][NT][4];
                score_tile<NT>(smem_u32(mem), smem_u32(ring.key_scales()), qf, s);
                if (there != 0xffffffffu || tok + kSub > least)
                    mask_tile<NT>(s, there, tok, end);
                float v[4] = {};
                #pragma unroll
                for (int n = 0; n < NT; ++n)
                    #pragma unroll
                    for (int i = 0; i < 4; ++i)
                        #pragma unroll
                        for (int x = 0; x < 2; ++x)
                            v[i] += ex2(fmaf(s[i >> 1][n][2 * (i & 1) + x], slc[n][x], z[n][x]));
                // the quad's lanes hold two columns of each eight: a lane ends with one of the
                // four tokens
                float w[2];
                #pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float give = c & 1 ? v[2 * i] : v[2 * i + 1];
                    w[i] = (c & 1 ? v[2 * i + 1] : v[2 * i]) + __shfl_xor_sync(0xffffffffu, give, 1);
                }
                const float give = c & 2 ? w[0] : w[1];
                const float sum = (c & 2 ? w[1] : w[0]) + __shfl_xor_sync(0xffffffffu, give, 2);
                if (mine < upto)
                    out[mine] = before + sum;
            }
            cp_async_wait<0>();
            __syncwarp();
        }
    }
    // ---- columns past the contexts, sixteen a lane at once
    if (a.mass == a.mass_out)
        return;
    constexpr int kEach = 16, kChunk = 32 * kEach;
    const int chunks = (a.width + kChunk - 1) / kChunk;
    const int64_t all = (int64_t)a.B * heads * chunks, step = (int64_t)gridDim.x * kGroups * kWarps;
    for (int64_t i = (int64_t)blockIdx.x * kGroups * kWarps + all_warp; i < all; i += step) {
        const int bh = (int)(i / chunks), at = (int)(i - (int64_t)bh * chunks) * kChunk;
        const int b = bh / heads, head = bh - b * heads, len = unit_len<true>(a, b);
        if (at + kChunk <= len)
            continue;
        const float *mass = a.mass ? a.mass + b * a.ld_batch + head * a.ld_head : nullptr;
        float *out = a.mass_out + b * a.ldo_batch + head * a.ldo_mass_head;
        float v[kEach];
        #pragma unroll
        for (int x = 0; x < kEach; ++x) {
            const int t = at + 32 * x + lane;
            v[x] = mass && t >= len && t < a.width ? mass[t] : 0.0f;
        }
        #pragma unroll
        for (int x = 0; x < kEach; ++x) {
            const int t = at + 32 * x + lane;
            if (t >= len && t < a.width)
                out[t] = v[x];
        }
    }
}

// ---------------------------------------------------------------------- host

// Columns of a block, in eights (32 sequences of 4 key heads: 32 columns as two
// blocks of 16 182 us, as one of 32, which spills, 189; 24 180 and 186).
int tiles_of(int cols)
{
    return cols <= 8 ? 1 : 2;
}

int groups_of(int nt)
{
    return nt == 1 ? Shape<1>::kGroups : Shape<2>::kGroups;
}

int part_of(int nt)
{
    return nt == 1 ? Shape<1>::kPart : Shape<2>::kPart;
}

// CTAs of a team for so many units of at most so many tiles: enough for a tile a group,
// as far as the SMs go; 0 where groups would have too many, or all tiles are so few
// that their pieces are joined sooner than a cluster starts (us, list and teams: 28
// tiles 8.4 and 9.3, 256 11.5 and 11.1, 512 14.6 and 13.0, 648 14.5 and 11.8; one to
// three sequences).  Of ragged slots the host knows the list's length, not its rows', and
// takes that for the longest: batches of rows mostly go without teams.
int team_of(int64_t units, int64_t tiles, int nt)
{
    const int sms = sm_count(), groups = groups_of(nt);
    if (units > sms || units * tiles < kTeamLeast)
        return 0;
    int team = 1;
    while (team < kTeamMost && 2 * team * units <= sms && tiles > (int64_t)team * groups)
        team *= 2;
    return tiles <= (int64_t)kTeamTiles * team * groups ? team : 0;
}

size_t cut_bytes(int shares)
{
    return ((size_t)shares * sizeof(int4) + 255) / 256 * 256;
}

// A kernel's shared memory is raised once a device.
template <typename F>
bool raise_smem(F kernel, int smem, std::atomic<uint64_t> &ready)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return false;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
            cudaSuccess)
            return false;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return true;
}

template <int kMode, int NT>
idx_status launch_team(const Kv4Args &a, cudaStream_t stream)
{
    constexpr int smem = Shape<NT>::template smem<kMode>();
    static std::atomic<uint64_t> ready{0};
    if (!raise_smem(kv4_attention_kernel<kMode, NT, true, false>, smem, ready))
        return IDX_ERR_CUDA;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.team;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * a.pool.heads * a.blocks * a.team));
    cfg.blockDim = dim3(Shape<NT>::kGroups * kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launch_status(cudaLaunchKernelEx(&cfg, kv4_attention_kernel<kMode, NT, true, false>, a));
}

template <int kMode, int NT>
idx_status launch_attention(Kv4Args &a, int64_t tiles, cudaStream_t stream)
{
    constexpr int smem = Shape<NT>::template smem<kMode>();
    static_assert(smem <= 226 * 1024, "shared memory of a CTA");
    if (a.team)
        return launch_team<kMode, NT>(a, stream);
    static std::atomic<uint64_t> ready[2]{};
    const bool listed = kMode == kSlots && a.uncut;
    const auto kernel = listed ? kv4_attention_kernel<kMode, NT, false, kMode == kSlots>
                               : kv4_attention_kernel<kMode, NT, false, false>;
    if (!raise_smem(kernel, smem, ready[listed]))
        return IDX_ERR_CUDA;
    const int64_t units = (int64_t)a.B * a.pool.heads * a.blocks;
    const int ctas = (int)std::min<int64_t>(sm_count(), tiles);
    const int shares = ctas * Shape<NT>::kGroups;
    a.by_unit = units < shares;
    cudaError_t e = launch_pdl(kernel, dim3(ctas),
                               dim3(Shape<NT>::kGroups * kThreads), smem, stream, a);
    if (e == cudaSuccess && !a.uncut) {
        // many pieces of few units: a block's warps share a column's
        const int cols = std::min(a.cols, 8 * NT), warps = kJoinThreads / 32;
        const int together = units * kJoinFew < shares;
        const int entries = a.by_unit ? (int)units : shares - 1;
        e = launch_pdl(kv4_join_kernel, dim3(entries, together ? cols : (cols + warps - 1) / warps),
                       dim3(kJoinThreads), 0, stream, a, 8 * NT, together);
    }
    return launch_status(e);
}

template <int kMode, int NT>
idx_status launch_weights(const Kv4Args &a, int64_t tiles, cudaStream_t stream)
{
    constexpr int smem = WeightShape<NT>::template smem<kMode>();
    static_assert(smem <= 226 * 1024, "shared memory of a CTA");
    static std::atomic<uint64_t> ready{0};
    if (!raise_smem(kv4_weights_kernel<kMode, NT>, smem, ready))
        return IDX_ERR_CUDA;
    return launch_status(launch_pdl(kv4_weights_kernel<kMode, NT>,
                                    dim3((int)std::min<int64_t>(sm_count(), tiles)),
                                    dim3(WeightShape<NT>::kGroups * kThreads), smem, stream, a));
}

// Checks that the calls share; keys: of a row at most.
idx_status check_attention(const void *q, int64_t ldq_row, int64_t ldq_head, int H, int kv_heads,
                           int D, float scale)
{
    if (!q || !(scale > 0.0f) || !(scale * kLog2e <= 3.4e38f) || ldq_head < D || ldq_row < 0)
        return IDX_ERR_INVALID_ARG;
    if (H % kv_heads != 0 || D != kKv4Dim || !aligned16(q) || (ldq_row | ldq_head) % 8 != 0)
        return IDX_ERR_UNSUPPORTED;
    return IDX_OK;
}

template <int kMode>
idx_status launch_columns(Kv4Args &a, int nt, int64_t tiles, cudaStream_t s)
{
    return nt == 1 ? launch_attention<kMode, 1>(a, tiles, s) : launch_attention<kMode, 2>(a, tiles, s);
}

// Fills in what a launch needs and launches.
template <bool kPaged>
idx_status run_attention(Kv4Args &a, int64_t keys, int64_t most_tiles, void *ws, size_t ws_bytes,
                         int H, idx_stream_t stream)
{
    const int nt = tiles_of(a.cols);
    a.blocks = (a.cols + 8 * nt - 1) / (8 * nt);
    const int64_t units = (int64_t)a.B * a.pool.heads * a.blocks;
    a.team = team_of(units, (keys + kTile - 1) / kTile, nt);
    a.uncut = !a.team && keys <= kUncutKeys;
    const int64_t tiles = a.uncut ? units : most_tiles * a.pool.heads * a.blocks;
    if ((int64_t)a.pool.heads * a.blocks > INT32_MAX / 2 || most_tiles > INT32_MAX / ((int64_t)a.pool.heads * a.blocks))
        return IDX_ERR_UNSUPPORTED;
    const size_t need = idx_kv4_attention_workspace_size(a.B * a.next_n, a.next_n, H, a.pool.heads, keys);
    if (need > 0 && (!ws || !aligned16(ws) || ws_bytes < need))
        return IDX_ERR_WORKSPACE;
    a.status = device_status_ptr();
    if (!a.status)
        return IDX_ERR_CUDA;
    const int most = sm_count() * groups_of(nt);
    a.ws_cut = static_cast<int4 *>(ws);
    a.ws_part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + cut_bytes(most));
    const cudaStream_t s = (cudaStream_t)stream;
    if constexpr (!kPaged)
        return launch_columns<kSlots>(a, nt, tiles, s);
    return a.pool.p.page_size % kSub == 0 ? launch_columns<kWholePages>(a, nt, tiles, s)
                                          : launch_columns<kPages>(a, nt, tiles, s);
}

} // namespace
} // namespace idx

using namespace idx;

extern "C" size_t idx_kv4_attention_workspace_size(int R, int next_n, int H, int kv_heads,
                                                   int64_t max_keys)
{
    if (R <= 0 || next_n <= 0 || H <= 0 || kv_heads <= 0 || max_keys <= kUncutKeys)
        return 0;
    const int64_t cols = (int64_t)next_n * (H / kv_heads);
    const int nt = tiles_of((int)std::min<int64_t>(cols, 32)), most = sm_count() * groups_of(nt);
    const int64_t units = (int64_t)(R / next_n) * kv_heads * ((cols + 8 * nt - 1) / (8 * nt));
    if (team_of(units, (max_keys + kTile - 1) / kTile, nt))
        return 0;
    return cut_bytes(most) + (size_t)2 * most * part_of(nt) * sizeof(float);
}

extern "C" idx_status idx_kv4_attention(const uint16_t *q, int64_t ldq_row, int64_t ldq_head,
                                        const uint8_t *kv_pages, int64_t page_stride_bytes,
                                        int num_pages, int page_size, const int32_t *slots,
                                        const int32_t *indptr, int64_t num_slots, int R, int H,
                                        int kv_heads, int D, float scale, uint16_t *out,
                                        int64_t ldo_row, int64_t ldo_head, float *lse,
                                        int64_t ld_lse, void *ws, size_t ws_bytes,
                                        idx_stream_t stream)
{
    IDX_NVTX_RANGE("idx_kv4_attention");
    if (R < 0 || H <= 0 || kv_heads <= 0 || D <= 0 || num_slots < 0)
        return IDX_ERR_INVALID_ARG;
    if (R == 0)
        return IDX_OK;
    if (!indptr || (num_slots > 0 && !slots) || !out || ldo_head < D || ldo_row < 0 ||
        (lse && ld_lse < H))
        return IDX_ERR_INVALID_ARG;
    idx_status ok = check_attention(q, ldq_row, ldq_head, H, kv_heads, D, scale);
    if (ok == IDX_OK)
        ok = check_kv4_pool(kv_pages, page_stride_bytes, num_pages, page_size, kv_heads);
    if (ok != IDX_OK)
        return ok;
    if (!aligned16(out) || (ldo_row | ldo_head) % 8 != 0 || num_slots > INT32_MAX - 4 * kTile)
        return IDX_ERR_UNSUPPORTED;
    if (!lie_apart({out, R, ldo_row, H, ldo_head, D, 2}))
        return IDX_ERR_INVALID_ARG;
    Kv4Args a = {};
    a.q = q;
    a.ldq_row = ldq_row;
    a.ldq_head = ldq_head;
    a.pool = make_kv4_pool(kv_pages, page_stride_bytes, num_pages, page_size, kv_heads);
    a.group = a.cols = H / kv_heads;
    a.next_n = 1;
    a.slots = slots;
    a.indptr = indptr;
    a.num_slots = num_slots;
    a.B = R;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.ldo_row = ldo_row;
    a.ldo_head = ldo_head;
    a.lse = lse;
    a.ld_lse = ld_lse;
    return run_attention<false>(a, num_slots, num_slots / kTile + R, ws, ws_bytes, H, stream);
}

extern "C" idx_status idx_paged_kv4_attention(
    const uint16_t *q, int64_t ldq_row, int64_t ldq_head, const uint8_t *kv_pages,
    int64_t page_stride_bytes, int num_pages, int page_size, const int32_t *block_table,
    int64_t bt_stride, const int32_t *context_lens, int ctx_per_row, int B, int next_n,
    int max_model_len, int H, int kv_heads, int D, float scale, uint16_t *out, int64_t ldo_row,
    int64_t ldo_head, float *lse, int64_t ld_lse, void *ws, size_t ws_bytes, idx_stream_t stream)
{
    IDX_NVTX_RANGE("idx_paged_kv4_attention");
    if (B < 0 || next_n <= 0 || H <= 0 || kv_heads <= 0 || D <= 0 || max_model_len < 0)
        return IDX_ERR_INVALID_ARG;
    if (B == 0)
        return IDX_OK;
    if (!context_lens || (max_model_len > 0 && !block_table) || !out || ldo_head < D ||
        ldo_row < 0 || (lse && ld_lse < H))
        return IDX_ERR_INVALID_ARG;
    idx_status ok = check_attention(q, ldq_row, ldq_head, H, kv_heads, D, scale);
    if (ok == IDX_OK)
        ok = check_kv4_pool(kv_pages, page_stride_bytes, num_pages, page_size, kv_heads);
    if (ok != IDX_OK)
        return ok;
    if (bt_stride < ((int64_t)max_model_len + page_size - 1) / page_size)
        return IDX_ERR_INVALID_ARG;
    const int64_t cols = (int64_t)next_n * (H / kv_heads);
    if (!aligned16(out) || (ldo_row | ldo_head) % 8 != 0 || cols > INT32_MAX / 2 ||
        (int64_t)B * next_n > INT32_MAX || max_model_len > INT32_MAX - 4 * kTile)
        return IDX_ERR_UNSUPPORTED;
    if (!lie_apart({out, (int64_t)B * next_n, ldo_row, H, ldo_head, D, 2}))
        return IDX_ERR_INVALID_ARG;
    Kv4Args a = {};
    a.q = q;
    a.ldq_row = ldq_row;
    a.ldq_head = ldq_head;
    a.pool = make_kv4_pool(kv_pages, page_stride_bytes, num_pages, page_size, kv_heads);
    a.group = H / kv_heads;
    a.cols = (int)cols;
    a.next_n = next_n;
    a.table = block_table;
    a.bt_stride = bt_stride;
    a.ctx = context_lens;
    a.ctx_per_row = ctx_per_row != 0;
    a.max_len = max_model_len;
    a.B = B;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.ldo_row = ldo_row;
    a.ldo_head = ldo_head;
    a.lse = lse;
    a.ld_lse = ld_lse;
    const int64_t tiles = std::max<int64_t>(1, ((int64_t)max_model_len + kTile - 1) / kTile);
    return run_attention<true>(a, max_model_len, B * tiles, ws, ws_bytes, H, stream);
}

extern "C" idx_status idx_paged_kv4_weights(
    const uint16_t *q, int64_t ldq_row, int64_t ldq_head, const uint8_t *kv_pages,
    int64_t page_stride_bytes, int num_pages, int page_size, const int32_t *block_table,
    int64_t bt_stride, const int32_t *context_lens, int ctx_per_row, int B, int next_n,
    int max_model_len, int H, int kv_heads, int D, float scale, const float *lse, int64_t ld_lse,
    int64_t ld_lse_head, const float *mass, int64_t ld_batch, int64_t ld_head, int width, float *out, int64_t ldo_batch,
    int64_t ldo_head, idx_stream_t stream)
{
    IDX_NVTX_RANGE("idx_paged_kv4_weights");
    if (B < 0 || next_n <= 0 || H <= 0 || kv_heads <= 0 || D <= 0 || max_model_len < 0 ||
        width < max_model_len)
        return IDX_ERR_INVALID_ARG;
    if (B == 0 || width == 0)
        return IDX_OK;
    if (!context_lens || (max_model_len > 0 && !block_table) || !lse || ld_lse < 0 || ld_lse_head < 0 || !out ||
        ld_batch < 0 || ld_head < 0 || ldo_batch < 0 || ldo_head < 0)
        return IDX_ERR_INVALID_ARG;
    idx_status ok = check_attention(q, ldq_row, ldq_head, H, kv_heads, D, scale);
    if (ok == IDX_OK)
        ok = check_kv4_pool(kv_pages, page_stride_bytes, num_pages, page_size, kv_heads);
    if (ok != IDX_OK)
        return ok;
    if (bt_stride < ((int64_t)max_model_len + page_size - 1) / page_size ||
        (mass == out && (ld_batch != ldo_batch || ld_head != ldo_head)))
        return IDX_ERR_INVALID_ARG;
    const int64_t cols = (int64_t)next_n * (H / kv_heads);
    const int64_t tiles = std::max<int64_t>(1, ((int64_t)max_model_len + kTile - 1) / kTile) * B;
    if (cols > INT32_MAX / 2 || (int64_t)B * next_n > INT32_MAX || width > INT32_MAX - 4 * kTile ||
        kv_heads > INT32_MAX / 2 || tiles > INT32_MAX / kv_heads)
        return IDX_ERR_UNSUPPORTED;
    const Strided sums = {out, B, ldo_batch, kv_heads, ldo_head, width, 4};
    if (!lie_apart(sums) ||
        (mass && mass != out && !lie_apart(sums, {mass, B, ld_batch, kv_heads, ld_head, width, 4})))
        return IDX_ERR_INVALID_ARG;
    Kv4Args a = {};
    a.q = q;
    a.ldq_row = ldq_row;
    a.ldq_head = ldq_head;
    a.pool = make_kv4_pool(kv_pages, page_stride_bytes, num_pages, page_size, kv_heads);
    a.group = H / kv_heads;
    a.cols = (int)cols;
    a.next_n = next_n;
    a.table = block_table;
    a.bt_stride = bt_stride;
    a.ctx = context_lens;
    a.ctx_per_row = ctx_per_row != 0;
    a.max_len = max_model_len;
    a.B = B;
    a.scale_log2 = scale * kLog2e;
    a.lse_in = lse;
    a.ld_lse_in = ld_lse;
    a.ld_lse_head = ld_lse_head;
    a.mass = mass;
    a.ld_batch = ld_batch;
    a.ld_head = ld_head;
    a.width = width;
    a.mass_out = out;
    a.ldo_batch = ldo_batch;
    a.ldo_mass_head = ldo_head;
    a.status = device_status_ptr();
    if (!a.status)
        return IDX_ERR_CUDA;
    // (without values there are registers for 32: 32 sequences of 4 key heads 111 us, as two
    // blocks 117)
    const int nt = a.cols <= 8 ? 1 : a.cols <= 16 ? 2 : 4;
    a.blocks = (a.cols + 8 * nt - 1) / (8 * nt);
    // the tiles of the contexts, and at least a warp for 512 columns past them
    const int64_t work = std::max<int64_t>(tiles * kv_heads,
                                           (int64_t)B * kv_heads * ((width + 511) / 512) / kWarps);
    const int mode = page_size % kSub == 0 ? kWholePages : kPages;
    const cudaStream_t st = (cudaStream_t)stream;
    return mode == kWholePages
               ? nt == 1 ? launch_weights<kWholePages, 1>(a, work, st)
                 : nt == 2 ? launch_weights<kWholePages, 2>(a, work, st)
                           : launch_weights<kWholePages, 4>(a, work, st)
               : nt == 1 ? launch_weights<kPages, 1>(a, work, st)
                 : nt == 2 ? launch_weights<kPages, 2>(a, work, st)
                           : launch_weights<kPages, 4>(a, work, st);
}
