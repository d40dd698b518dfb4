// idx_prefill.cuh -- attention of ragged sequences with keys and values of 128
// elements a head: out = softmax(scale * q . k) . v.  In the expanded form of
// latent attention (kRope) keys have 64 elements more, which all heads share; the
// grouped form has several query heads to a key head.  What follows is of the
// first, which takes three pieces of queries and keys; the second takes two.
//
// A block is up to two tiles of 128 queries of one head; a CTA walks the keys
// they see, 128 at a time, with a running maximum and sum:
//
//     S [128 queries x 128 keys] = Q [128 x 192] . K^T   (12 MMAs, 128 x 128 x 16)
//     O [128 x 128]             += P [128 x 128] . V     (2 x 8 MMAs, 128 x 64 x 16)
//
// The two tiles take turns: while the softmax warps of one work, the tensor
// cores do the other's products, and both read each key tile once.  Scores,
// weights and sums stay in tensor memory: S (128 columns) is overwritten by P
// in bf16, which the second product takes as its A operand from there.  Bounds:
// the tensor cores need 2610 cycles for both tiles' products with a key tile
// (12 of 65 and 16 of 33 each), a tile's softmax 1150, by its instructions
// (pairs of scores share them where they can; exponentials by polynomial beside
// the special-function unit's cost more of them and time).  Measured: 3030
// cycles; 2048 queries x 64 heads at the end of 8192 tokens 380 to 397 us in
// short bursts (1500 to 1580 TFLOP/s) and 432 to 444 in calls that go on, where
// the GPU's power limit holds it whatever the kernel saves; 7 whole prompts of
// 65 to 1500 tokens x 16 heads 55 us.
//
// Keys and values come by TMA in pieces of 64 elements of 128 tokens (16 KB,
// 128-byte swizzled), five a tile (three of K, the last shared by all heads,
// two of V), around a ring of eight places: K^T is read K-major, V M-major, as they
// lie.  The running maximum is only raised when a score exceeds it by 2^40
// (32-bit sums lose nothing by that), so rescaling O is rare after a row's
// first tile.
//
// Work is the flat list of (head, block, key tile); every CTA (one per SM)
// takes an equal contiguous share of it, so causal blocks of any length fill
// the GPU evenly and few queries on many keys are spread over it; a block
// counts a tile more than it has, for the end of the one before (the prompts
// 54.8 us; none 58.8, two 55.0).  The products go from block to block without a
// pause: a query tile's next scores follow its last values at once, in the next
// block while the other tile still works on this one (62.9 us with a pause), as
// its place and the keys' come free.  A block
// that shares cut leaves unnormalised sums in scratch for a second kernel.
//
// Warps: 0-3 and 4-7 softmax of the two tiles, a thread a query; 8 issues TMA;
// 9 issues the products; 10 clears values past a sequence's end.
#pragma once

#include <algorithm>
#include <atomic>
#include <cuda_bf16.h>

#include "idx_common.cuh"
#include "idx_internal.h"

namespace idx {
namespace {

constexpr int kV = 128;                         // elements of a head's keys and values
constexpr int kTile = 128;                      // queries and keys of a tile
constexpr int kPiece = kTile * 128;             // bytes of 64 elements of a tile's tokens
constexpr int kVPieces = kV / 64;
constexpr int kRing = 8;
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpTail = 10;
constexpr int kThreads = 384;  // whole warpgroups: the last warp only helps to start
// Registers of a thread: as launched, then of the two softmax warpgroups (a
// row of scores each thread) and of the third.
constexpr int kRegs = 168, kRegsSoft = 200, kRegsRest = 104;
static_assert(2 * kRegsSoft + kRegsRest <= 3 * kRegs && kRegs * kThreads <= 65536,
              "the warpgroups' registers come from the launch's");
constexpr int kBars = kRing + 20;
constexpr int kMaxCu = 128;

// Pieces of a tile and the layout of shared memory.
template <bool kRope>
struct Lay {
    static constexpr int kQPieces = kV / 64 + (kRope ? 1 : 0), kPieces = kQPieces + kVPieces;
    static constexpr int kOffRing = 2 * kQPieces * kPiece;
    static constexpr int kOffBar = kOffRing + kRing * kPiece;
    static constexpr int kOffMisc = kOffBar + 8 * kBars;  // tmem base, abort flag, the share's place, sizes
    static constexpr int kOffSum = kOffMisc + 32;         // a sum of each warp
    static constexpr int kOffCu = kOffSum + kThreads / 4; // the sequences' bounds, where they fit
    static constexpr int kSmem = kOffCu + 8 * (kMaxCu + 1) + 1024;  // the base is aligned to 1024
    static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};
constexpr uint32_t kColS = 0, kColO = 256;     // tensor memory columns, 128 a query tile
constexpr float kLazy = 40.0f;                 // a score may exceed its running maximum by 2^40
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

struct PrefillArgs {
    const int32_t *cu_q, *cu_k;
    int B, Tq, Tk, H;
    int group;       // query heads of a key head
    float scale_log2;
    int causal;
    __nv_bfloat16 *out;
    int64_t ldo_row, ldo_head;
    float *lse;
    int64_t ld_lse;
    int uncut;       // shares end with blocks: no partial results
    int4 *ws_cut;    // two a share: the block it begins and leaves to the next (head, sequence,
                     // block, pieces; no pieces: none), whether a segment lies before it
    float *ws_part;  // two segments a share: for each query tile O, maxima, sums
    unsigned int *status;
};

constexpr int kRows = 2 * kTile;                        // queries of a block
constexpr int kPartTile = kTile * kV + 2 * kTile;       // floats of a query tile's partial result
constexpr int kMaxShares = 152;
constexpr int kCharge = 1;  // tiles that a block counts besides its own
constexpr int64_t kMaxHeadTiles = (int64_t)1 << 36;  // of all heads: a share's fit 32 bits
// Blocks of few keys are not cut: up to four tiles a CTA more cost less than
// the joining kernel (6.6 us whole, 8.1 cut, for 2 sequences of 50 rows, 3
// heads).
constexpr int kUncutKeys = 4 * kTile;

// A block: queries kRows i .. of sequence b, for one head.
struct Block {
    int head, b, i;
    int seq_q, nq, seq_k, nk;
};

// The sequence's rows (bounds outside the tensors are clamped).
__device__ __forceinline__ void block_seq(const PrefillArgs &a, const int32_t *cq,
                                          const int32_t *ck, Block &k)
{
    k.seq_q = min(max(cq[k.b], 0), a.Tq);
    k.nq = max(0, min(cq[k.b + 1], a.Tq) - k.seq_q);
    k.seq_k = min(max(ck[k.b], 0), a.Tk);
    k.nk = max(0, min(ck[k.b + 1], a.Tk) - k.seq_k);
}

// The next block: of the sequence, of the next one that has queries, of the
// next head.  Only called when there is one.
__device__ __forceinline__ void block_next(const PrefillArgs &a, const int32_t *cq,
                                           const int32_t *ck, Block &k)
{
    ++k.i;
    while (k.i * kRows >= k.nq) {
        k.i = 0;
        if (++k.b == a.B) {
            k.b = 0;
            ++k.head;
        }
        block_seq(a, cq, ck, k);
    }
}

// Keys that query row r of the sequence sees.
__device__ __forceinline__ int keys_seen(const PrefillArgs &a, const Block &k, int r)
{
    return a.causal ? min(k.nk, max(0, r + k.nk - k.nq + 1)) : k.nk;
}

// Key tiles of query tile q of the block (0: it has no queries, or they no keys).
__device__ __forceinline__ int key_tiles(const PrefillArgs &a, const Block &k, int q)
{
    const int first = k.i * kRows + q * kTile, last = min(first + kTile, k.nq) - 1;
    return last < first ? 0 : (keys_seen(a, k, last) + kTile - 1) / kTile;
}

// Tiles of the first n blocks of a sequence, its last not among them; a block
// counts at least one, its outputs are written (causal: block i sees kRows /
// kTile (i + 1) + ceil((nk - nq) / kTile) tiles).  Lists are counted in 64
// bits, shares in 32.
__device__ __forceinline__ int64_t tiles_before(const PrefillArgs &a, int nq, int nk, int n)
{
    if (!a.causal)
        return (int64_t)n * max(1, (nk + kTile - 1) / kTile);
    constexpr int rho = kRows / kTile;
    const int d = nk - nq;
    const int delta = d >= 0 ? (d + kTile - 1) / kTile : -(-d / kTile);
    const int z = min(n, max(0, -delta / rho));  // blocks that see nothing
    return z + rho * ((int64_t)n * (n + 1) - (int64_t)z * (z + 1)) / 2 + (int64_t)delta * (n - z);
}

// All of a sequence's tiles and its blocks' charges: below 2^48.
__device__ __forceinline__ int64_t tiles_of_seq(const PrefillArgs &a, int nq, int nk)
{
    if (nq <= 0)
        return 0;
    const int blocks = (nq + kRows - 1) / kRows;
    return tiles_before(a, nq, nk, blocks - 1) + max(1, (nk + kTile - 1) / kTile) +
           blocks * kCharge;
}

// The walk of a share: segments of a block's tiles.
struct Walk {
    Block k;
    int t, left;  // left: tiles and charges
    int pay;      // of the block's charge
};

struct Seg {
    Block k;
    int t0, t1, tiles;
    int nt[2];  // unrolled uses only
};

__device__ __forceinline__ bool next_seg(const PrefillArgs &a, const int32_t *cq,
                                         const int32_t *ck, Walk &w, Seg &s)
{
    if (w.t < 0 && w.left > (a.uncut ? 0 : kCharge)) {
        block_next(a, cq, ck, w.k);
        w.t = 0;
        w.pay = kCharge;
    }
    if (w.left <= (a.uncut ? 0 : w.pay) || w.t < 0)
        return false;
    w.left -= w.pay;
    w.pay = 0;
    s.k = w.k;
    s.t0 = w.t;
    s.nt[0] = key_tiles(a, w.k, 0);
    s.nt[1] = key_tiles(a, w.k, 1);
    s.tiles = max(1, max(s.nt[0], s.nt[1]));
    s.t1 = a.uncut ? s.tiles : min(s.tiles, w.t + w.left);
    w.left -= s.t1 - s.t0;
    w.t = s.t1 < s.tiles ? s.t1 : -1;
    return true;
}

// Two bf16 of scaled sums.
__device__ __forceinline__ uint32_t pack2(uint32_t a, uint32_t b, float f)
{
    const __nv_bfloat162 v =
        __floats2bfloat162_rn(__uint_as_float(a) * f, __uint_as_float(b) * f);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// 4 x 4 words turned over among the four lanes of a quad: word x of lane c
// becomes word c of lane x.
__device__ __forceinline__ void turn_quad(uint32_t (&w)[4], int c)
{
    #pragma unroll
    for (int e = 0; e < 4; e += 2) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, c & 1 ? w[e] : w[e + 1], 1);
        w[e] = c & 1 ? got : w[e];
        w[e + 1] = c & 1 ? w[e + 1] : got;
    }
    #pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, c & 2 ? w[e] : w[e + 2], 2);
        w[e] = c & 2 ? got : w[e];
        w[e + 2] = c & 2 ? w[e + 2] : got;
    }
}

template <bool kRope>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_r,
                          const __grid_constant__ CUtensorMap tm_v, const PrefillArgs a)
{
    constexpr int kQPieces = Lay<kRope>::kQPieces, kPieces = Lay<kRope>::kPieces;
    constexpr int kOffRing = Lay<kRope>::kOffRing, kOffBar = Lay<kRope>::kOffBar;
    constexpr int kOffMisc = Lay<kRope>::kOffMisc, kOffSum = Lay<kRope>::kOffSum;
    constexpr int kOffCu = Lay<kRope>::kOffCu;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + kOffBar);
    // a piece of the ring came in; the keys and the values of even and odd tiles
    // were read by their last product
    uint64_t *full = bar, *k_free = bar + kRing, *v_free = k_free + 2;
    uint64_t *s_full = k_free + 4, *p_full = k_free + 6, *pv_done = k_free + 8;
    uint64_t *q_full = k_free + 10, *q_free = k_free + 12, *drain = k_free + 14;
    uint64_t *tail = k_free + 15;  // cut values came in: [even and odd cut tiles][pieces]
    int *misc = reinterpret_cast<int *>(smem + kOffMisc);
    volatile int *abort_flag = misc + 1;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

    if (tid == 0) {
        for (int i = 0; i < kRing; ++i)
            mbar_init(&full[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tail[2 * i], 1);
            mbar_init(&tail[2 * i + 1], 1);
            mbar_init(&k_free[i], 4);
            mbar_init(&v_free[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&pv_done[i], 1);
            mbar_init(&q_full[i], 1);
            mbar_init(&q_free[i], 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(reinterpret_cast<uint32_t *>(misc), 512);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_launch_dependents();

    // ---- this CTA's share: the tiles of a head are those of all sequences
    const int32_t *cq = a.cu_q, *ck = a.cu_k;
    if (a.B <= kMaxCu) {
        int32_t *cu = reinterpret_cast<int32_t *>(smem + kOffCu);
        for (int i = tid; i <= a.B; i += kThreads) {
            cu[i] = a.cu_q[i];
            cu[kMaxCu + 1 + i] = a.cu_k[i];
        }
        cq = cu;
        ck = cu + kMaxCu + 1;
    }
    __syncthreads();
    if (tid == 0 && !a.uncut)
        a.ws_cut[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    int64_t *wsum = reinterpret_cast<int64_t *>(smem + kOffSum);
    const auto seq_tiles = [&](int b) -> int64_t {
        Block k;
        k.b = b;
        if (b >= a.B)
            return 0;
        block_seq(a, cq, ck, k);
        if (blockIdx.x == 0 && (cq[b] < 0 || cq[b + 1] < cq[b] || cq[b + 1] > a.Tq || ck[b] < 0 ||
                                ck[b + 1] < ck[b] || ck[b + 1] > a.Tk))
            atomicOr(a.status, kDevBadBounds);
        return tiles_of_seq(a, k.nq, k.nk);
    };
    int64_t head_tiles = 0, mine, before;
    const auto scan = [&](int b0) {  // of sequences b0 + thread; adds up head_tiles
        mine = seq_tiles(b0 + tid);
        int64_t upto = mine;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? v : 0;
        }
        __syncthreads();
        if (lane == 31)
            wsum[warp] = upto;
        __syncthreads();
        before = head_tiles + upto - mine;
        #pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
            before += i < warp ? wsum[i] : 0;
            head_tiles += wsum[i];
        }
        head_tiles = min(head_tiles, kMaxHeadTiles);
    };
    for (int b0 = 0; b0 < a.B; b0 += kThreads)
        scan(b0);
    // A list that no device lives to the end of (of bounds that descend: its
    // sequences hold tokens again) is left alone.
    const bool too_many = head_tiles >= kMaxHeadTiles / a.H;
    if (too_many) {
        if (blockIdx.x == 0 && tid == 0)
            atomicOr(a.status, kDevBadBounds);
        head_tiles = 0;
    }
    const int64_t total = head_tiles * a.H;
    // two tiles a share at least: a cut costs about as much as a tile
    const int p = blockIdx.x, shares = (int)max((int64_t)1, min((int64_t)gridDim.x, total / 2));
    const int each = (int)(total / shares), more = (int)(total - (int64_t)each * shares);
    if (tid == 0) {
        misc[4] = each;
        misc[5] = more;
    }
    const int64_t u0 = (int64_t)p * each + min(p, more);
    Walk w;
    w.left = p < shares && total > 0 ? each + (p < more) : 0;
    w.k.head = w.left > 0 ? (int)(u0 / head_tiles) : 0;
    const int64_t at = u0 - w.k.head * head_tiles;
    int64_t *rest_at = reinterpret_cast<int64_t *>(misc + 2);
    if (a.B > kThreads && !too_many) {
        // many sequences: the chunk that holds the place, once more
        head_tiles = 0;
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            scan(b0);
            if (w.left > 0 && at >= before && at < before + mine) {
                misc[6] = b0 + tid;
                *rest_at = at - before;
            }
        }
    } else if (w.left > 0 && at >= before && at < before + mine) {
        misc[6] = tid;
        *rest_at = at - before;
    }
    __syncthreads();
    tc_fence_after();
    // one value for the warp, as the compiler sees it too
    const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);
    w.t = w.pay = 0;
    if (w.left > 0) {
        w.k.b = __shfl_sync(0xffffffffu, misc[6], 0);
        const int64_t place = __shfl_sync(0xffffffffu, *rest_at, 0);
        block_seq(a, cq, ck, w.k);
        int lo = 0, hi = (w.k.nq + kRows - 1) / kRows - 1;  // the last i with tiles_before <= rest
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (tiles_before(a, w.k.nq, w.k.nk, mid) + mid * kCharge <= place)
                lo = mid;
            else
                hi = mid - 1;
        }
        w.k.i = lo;
        const int rest = (int)(place - (tiles_before(a, w.k.nq, w.k.nk, lo) + lo * kCharge));
        w.t = max(0, rest - kCharge);
        w.pay = max(0, kCharge - rest);
        if (a.uncut && rest > 0) {
            // the share that the block begins in has all of it
            w.left -= kCharge - rest + max(1, max(key_tiles(a, w.k, 0), key_tiles(a, w.k, 1)));
            w.t = -1;
            w.pay = 0;
        }
    }
    Seg s;

    if (warp < kWarpLoad) {
        // ------------------------------------------------ softmax, epilogue
        regs_take<kRegsSoft>();
        const int q = warp >> 2;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t col_s = tmem + lanes + kColS + q * 128, col_o = tmem + lanes + kColO + q * 128;
        const float sl = a.scale_log2;
        int i = 0, n = 0, segs = 0;  // tiles of this query tile, of both, its segments so far
        Seg ahead;
        bool more = next_seg(a, cq, ck, w, s);
        for (int seg = 0; more; ++seg, s = ahead) {
            const int row = s.k.i * kRows + q * kTile + (tid & 127);
            // rows past the sequence's queries take part with no key
            const int seen = row < s.k.nq ? keys_seen(a, s.k, row) : 0;
            // the warp's fewest, if it has all its rows
            const int seen_first = __shfl_sync(0xffffffffu, seen, 0);
            const bool whole_warp = __all_sync(0xffffffffu, row < s.k.nq);
            const int t1 = min(s.t1, q ? s.nt[1] : s.nt[0]);
            float m = -INFINITY, l = 0.0f;
            for (int j = s.t0; j < t1; ++j, ++i) {
                // after an abort the waits return at once and the loop runs out
                (void)mbar_wait_here(&s_full[q], i & 1, abort_flag, a.status);
                __syncwarp();
                tc_fence_after();
                // the keys are free after the tile's last S, the queries after
                // the segment's
                if (lane == 0 && (q == 1 || s.nt[1] <= j))
                    mbar_arrive(&k_free[(n + j - s.t0) & 1]);
                if (lane == 0 && j + 1 == t1)
                    mbar_arrive(&q_free[q]);
                uint32_t r[4][32];
                #pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld_32x32b_x32(col_s + 32 * c, r[c]);
                tmem_ld_wait();
                if (!whole_warp || (j + 1) * kTile > seen_first) {
                    const int lim = seen - j * kTile;
                    #pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        #pragma unroll
                        for (int e = 0; e < 32; ++e)
                            r[c][e] = 32 * c + e < lim ? r[c][e] : 0xff800000u;
                    }
                }
                float mx[4];
                #pragma unroll
                for (int c = 0; c < 4; ++c) {
                    mx[c] = __uint_as_float(r[c][0]);
                    #pragma unroll
                    for (int e = 1; e < 32; ++e)
                        mx[c] = fmaxf(mx[c], __uint_as_float(r[c][e]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl;
                // -inf - -inf (no key so far) is no reason to raise it
                if (__any_sync(0xffffffffu, top - m > kLazy)) {
                    const float nm = fmaxf(m, top);
                    const float al = nm == m ? 1.0f : ex2(m - nm);
                    m = nm;
                    l *= al;
                    if (j > s.t0) {
                        // O is complete: S was issued after its last product, and
                        // a commit covers all that its thread issued before
                        #pragma unroll 1
                        for (int c = 0; c < 128; c += 16) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16(col_o + c, o);
                            tmem_ld_wait();
                            #pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                            tmem_st_32x32b_x16(col_o + c, o);
                        }
                        tmem_st_wait();
                    }
                }
                const float nm = m == -INFINITY ? 0.0f : -m;
                const uint64_t sl2 = pack_x2(sl, sl), nm2 = pack_x2(nm, nm);
                uint64_t sum[2] = {};
                #pragma unroll
                for (int c = 0; c < 2; ++c) {
                    // weights as bf16 (half a step of 2^-8 each), two a column
                    uint32_t v[32];
                    #pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint32_t *at = &r[2 * c + (e >> 4)][2 * e & 31];
                        const uint64_t x = ex2_x2(fma_x2(pack_x2(at[0], at[1]), sl2, nm2));
                        sum[e & 1] = add_x2(sum[e & 1], x);
                        const __nv_bfloat162 b2 = __floats2bfloat162_rn(low_x2(x), high_x2(x));
                        v[e] = *reinterpret_cast<const uint32_t *>(&b2);
                    }
                    tmem_st_32x32b_x32(col_s + 32 * c, v);
                }
                sum[0] = add_x2(sum[0], sum[1]);
                l += low_x2(sum[0]) + high_x2(sum[0]);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&p_full[q]);
            }
            // ---- the segment's sums
            const bool some = t1 > s.t0;
            n += max(0, min(s.t1, max(s.nt[0], s.nt[1])) - s.t0);
            more = next_seg(a, cq, ck, w, ahead);  // while the last products run
            if (some) {
                (void)mbar_wait_here(&pv_done[q], segs & 1, abort_flag, a.status);
                ++segs;
                __syncwarp();
                tc_fence_after();
            }
            if (s.t0 > 0 || s.t1 < s.tiles) {
                // a part of the block: scratch, rows side by side
                float *part = a.ws_part + ((int64_t)(2 * blockIdx.x + (seg > 0)) * 2 + q) * kPartTile;
                const int r4 = 4 * (tid & 127);
                if (some) {
                    #pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(col_o + c, o);
                        tmem_ld_wait();
                        #pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<uint4 *>(part + (c + e) * kTile + r4) =
                                make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                if (tid == 0 && s.t0 == 0) {
                    // the shares that hold the rest: `more - p - 1` longer ones first
                    const int size = misc[4], longer = max(0, misc[5] - (int)blockIdx.x - 1);
                    const int rest = s.tiles - s.t1;
                    const int in = (int)min((int64_t)rest, (int64_t)longer * (size + 1));
                    a.ws_cut[2 * blockIdx.x] = make_int4(
                        s.k.head, s.k.b, s.k.i,
                        1 + (in + size) / (size + 1) + (rest - in + size - 1) / size);
                    a.ws_cut[2 * blockIdx.x + 1] = make_int4(seg > 0, 0, 0, 0);
                }
                part[kTile * kV + (tid & 127)] = m;
                part[kTile * kV + kTile + (tid & 127)] = l;
            } else if (__any_sync(0xffffffffu, row < s.k.nq)) {
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                if (a.lse && row < s.k.nq)
                    a.lse[(int64_t)(s.k.seq_q + row) * a.ld_lse + s.k.head] =
                        l == 0.0f ? -INFINITY : ((m == -INFINITY ? 0.0f : m) + log2f(l)) * kLn2;
                // rows g, g + 8 of each half warp's sixteen; a quad of lanes
                // holds 64 contiguous bytes of each after turning over
                const int g = lane >> 2, c4 = lane & 3;
                __nv_bfloat16 *to = a.out + (int64_t)s.k.seq_q * a.ldo_row +
                                    s.k.head * a.ldo_head + 8 * c4;
                const int row0 = row - lane;
                #pragma unroll 1
                for (int hc = 0; hc < 4; ++hc) {
                    const int half = hc >> 1, c0 = 64 * (hc & 1);
                    uint32_t o[32];
                    #pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = 0;
                    if (some) {
                        tmem_ld_16x256b<8>(col_o + ((uint32_t)(16 * half) << 16) + c0, o);
                        tmem_ld_wait();
                    }
                    #pragma unroll
                    for (int up = 0; up < 2; ++up) {
                        const int r = row0 + 16 * half + 8 * up + g;
                        const float f = __shfl_sync(0xffffffffu, inv, 16 * half + 8 * up + g);
                        #pragma unroll
                        for (int x = 0; x < 8; x += 4) {
                            uint32_t v[4];
                            #pragma unroll
                            for (int e = 0; e < 4; ++e)
                                v[e] = pack2(o[4 * (x + e) + 2 * up], o[4 * (x + e) + 2 * up + 1], f);
                            turn_quad(v, c4);
                            if (r < s.k.nq)
                                *reinterpret_cast<uint4 *>(to + (int64_t)r * a.ldo_row + c0 +
                                                           8 * x) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    }
                }
            }
            tc_fence_before();
        }
    } else if (regs_give<kRegsRest>(), warp == kWarpLoad) {
        // ------------------------------------------------------------- TMA
        const bool one = elect_one();
        int n = 0, pieces = 0;    // tiles and pieces issued
        int tails = 0;            // tiles whose values a sequence's end cuts
        int loads[2] = {0, 0};    // of each query tile
        bool ok = true;
        while (ok && next_seg(a, cq, ck, w, s)) {
            // Query tile 0's queries, the first keys, tile 1's queries, the first
            // values: in the order in which the segment before frees their places.
            const auto queries = [&](int q) {
                // the last segment's products have read the ones before
                if (loads[q] > 0)
                    ok = mbar_wait_here(&q_free[q], (loads[q] - 1) & 1, abort_flag, a.status);
                if (!ok)
                    return;
                __syncwarp();
                if (one) {
                    mbar_arrive_expect_tx(&q_full[q], kQPieces * kPiece);
                    #pragma unroll 1
                    for (int c = 0; c < kQPieces; ++c)
                        tma_load_3d(smem + (q * kQPieces + c) * kPiece, &tm_q, &q_full[q], 128 * c,
                                    s.k.head, s.k.seq_q + s.k.i * kRows + q * kTile);
                }
                ++loads[q];
            };
            const int key_head = kRope ? s.k.head : s.k.head / a.group;
            if (s.nt[0] > s.t0)
                queries(0);
            const int most = min(s.t1, max(s.nt[0], s.nt[1]));
            for (int j = s.t0; ok && j < most; ++j, ++n) {
                const int t0 = s.k.seq_k + j * kTile, rem = s.k.nk - j * kTile;
                const bool cut = rem < kTile;  // values past the sequence
                #pragma unroll 1
                for (int c = 0; ok && c < kPieces; ++c) {
                    // Of five pieces, 5 n + c takes the place of 5 n + c - 8: the last of
                    // tile n - 2's keys (c = 0), its values (1, 2), tile n - 1's first keys
                    // (3, 4).  Of four, the place of its like in tile n - 2.
                    const int m = n * kPieces + c, slot = m & (kRing - 1);
                    if (c == kQPieces && j == s.t0 && s.nt[1] > s.t0) {
                        queries(1);
                        if (!ok)
                            break;
                    }
                    if (c == 0 && n >= 2)
                        ok = mbar_wait_here(&k_free[n & 1], ((n >> 1) - 1) & 1, abort_flag,
                                            a.status);
                    else if (c == (kRope ? 1 : kQPieces) && n >= 2)
                        ok = mbar_wait_here(&v_free[n & 1], ((n >> 1) - 1) & 1, abort_flag,
                                            a.status);
                    else if (kRope && c == kQPieces && n >= 1)
                        ok = mbar_wait_here(&k_free[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag,
                                            a.status);
                    if (!ok)
                        break;
                    __syncwarp();
                    uint8_t *to = smem + kOffRing + slot * kPiece;
                    if (one) {
                        uint64_t *b = cut && c >= kQPieces ? &tail[2 * (tails & 1) + c - kQPieces]
                                                           : &full[slot];
                        mbar_arrive_expect_tx(b, kPiece);
                        if (c < 2)
                            tma_load_3d(to, &tm_k, b, 128 * c, key_head, t0);
                        else if (kRope && c == 2)
                            tma_load_2d(to, &tm_r, b, 0, t0);
                        else
                            tma_load_3d(to, &tm_v, b, 128 * (c - kQPieces), key_head, t0);
                    }
                    pieces = m + 1;
                }
                tails += cut && ok;
            }
        }
        if (*abort_flag) {
            // the copies in flight land before the CTA leaves
            #pragma unroll
            for (int q = 0; q < 2; ++q)
                if (loads[q] > 0)
                    (void)mbar_drain_here(&q_full[q], (loads[q] - 1) & 1);
            for (int t = max(0, tails - 2); t < tails; ++t)
                for (int c = 0; c < kVPieces; ++c)
                    (void)mbar_drain_here(&tail[2 * (t & 1) + c], (t >> 1) & 1);
            for (int i = max(0, pieces - kRing); i < pieces; ++i)
                (void)mbar_drain_here(&full[i & (kRing - 1)], (i >> 3) & 1);
        }
    } else if (warp == kWarpMma) {
        // ------------------------------------------------------------ MMAs
        const uint32_t one = elect_one();
        const uint32_t id_s = idesc_bf16(kTile, kTile, false, false);
        const uint32_t id_v = idesc_bf16(kTile, 64, false, true);
        int n0 = -1;           // tiles before the segment
        int fills = 0;         // parity of the segments that each query tile had, a bit each
        int done0 = 0, done1 = 0;  // tiles of each query tile before the segment
        // S of query tile q and the segment's k-th key tile.  Commits cost the
        // issuing warp about a hundred cycles each: there are no more than needed.
        const auto scores = [&](int q, int k, bool first) {
            const int n = n0 + k, slot = n * kPieces;
            const uint32_t qd = desc_lo(sbase + q * kQPieces * kPiece);
            #pragma unroll
            for (int c = 0; c < kQPieces; ++c) {
                const int m = slot + c;
                if (first && !mbar_wait_here(&full[m & (kRing - 1)], (m >> 3) & 1, abort_flag,
                                             a.status))
                    return false;
                __syncwarp();
                tc_fence_after();
                const uint32_t kd = desc_lo(sbase + kOffRing + (m & (kRing - 1)) * kPiece);
                #pragma unroll
                for (int e = 0; e < 4; ++e)
                    mma_f16(tmem + kColS + q * 128, qd + (c * kPiece >> 4) + 2 * e, kd + 2 * e,
                            kDescHiSw128, id_s, c + e > 0 ? 1u : 0u, one);
            }
            mma_commit_if(&s_full[q], one);
            return true;
        };
        // O += P V; the last query tile of a key tile frees its values
        const auto values = [&](int q, int k, int done, bool first, bool last, bool end) {
            const int n = n0 + k, slot = n * kPieces + kQPieces;
            if (!mbar_wait_here(&p_full[q], (done + k) & 1, abort_flag, a.status))
                return false;
            #pragma unroll
            for (int c = 0; c < kVPieces; ++c) {
                const int m = slot + c;
                if (first && !mbar_wait_here(&full[m & (kRing - 1)], (m >> 3) & 1, abort_flag,
                                             a.status))
                    return false;
                __syncwarp();
                tc_fence_after();
                const uint32_t vd = desc_lo(sbase + kOffRing + (m & (kRing - 1)) * kPiece);
                #pragma unroll
                for (int e = 0; e < 8; ++e)
                    mma_f16_ts(tmem + kColO + q * 128 + 64 * c, tmem + kColS + q * 128 + 8 * e,
                               vd + e * (2048 >> 4), kDescHiSw128, id_v, k + e > 0 ? 1u : 0u, one);
            }
            if (last)
                mma_commit_if(&v_free[n & 1], one);
            if (end)
                mma_commit_if(&pv_done[q], one);
            return true;
        };
        // Tile by tile: its products of each query tile, each followed by the next
        // tile's scores of the same one, in the next segment as in this.  Before
        // the first segment stands one of a tile that none takes.
        int c0 = 0, c1 = 0;  // the segment's tiles for each query tile
        bool ok = true, more = true;
        while (ok && more) {
            int x0 = 0, x1 = 0;  // the next segment's
            while (max(x0, x1) == 0 && (more = next_seg(a, cq, ck, w, s))) {
                x0 = max(0, min(s.t1, s.nt[0]) - s.t0);
                x1 = max(0, min(s.t1, s.nt[1]) - s.t0);
            }
            const int most = max(1, max(c0, c1));
            #pragma unroll 1
            for (int k = 0; ok && k < most; ++k) {
                const bool last = k + 1 == most;
                #pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int cnt = q ? c1 : c0;
                    if (ok && k < cnt)
                        ok = values(q, k, q ? done1 : done0, q == 0 || c0 <= k, q == 1 || c1 <= k,
                                    k + 1 == cnt);
                    const bool fresh = last && (q ? x1 : x0) > 0;
                    if (ok && fresh) {
                        ok = mbar_wait_here(&q_full[q], (fills >> q) & 1, abort_flag, a.status);
                        fills ^= 1 << q;
                    }
                    if (ok && (fresh || k + 1 < cnt))
                        ok = scores(q, k + 1, q == 0 || (last ? x0 : c0 - k - 1) <= 0);
                }
            }
            n0 += most;
            done0 += c0;
            done1 += c1;
            c0 = x0;
            c1 = x1;
        }
        if (*abort_flag) {
            mma_commit_if(drain, one);
            __syncwarp();
            (void)mbar_drain_here(drain, 0);
        }
    }
    else if (warp == kWarpTail) {
        // ---------------------------------------------- values of a cut tile
        // A weight of zero does not hide what is not finite: another sequence's
        // values become zeros here.
        int n = 0, tails = 0;
        bool ok = true;
        while (ok && next_seg(a, cq, ck, w, s)) {
            const int most = min(s.t1, max(s.nt[0], s.nt[1]));
            const int j = s.k.nk / kTile, rem = s.k.nk % kTile;
            if (rem > 0 && j >= s.t0 && j < most) {
                #pragma unroll 1
                for (int c = 0; c < kVPieces; ++c) {
                    ok = mbar_wait_here(&tail[2 * (tails & 1) + c], (tails >> 1) & 1, abort_flag,
                                        a.status);
                    if (!ok)
                        break;
                    const int slot = ((n + j - s.t0) * kPieces + kQPieces + c) & (kRing - 1);
                    const uint32_t to = smem_u32(smem + kOffRing + slot * kPiece);
                    #pragma unroll 1
                    for (int e = rem * 8 + lane; e < kTile * 8; e += 32)
                        st_shared_v4(to + 16 * e, 0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&full[slot]);
                }
                ++tails;
            }
            n += max(0, most - s.t0);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma)
        tmem_dealloc(tmem, 512);
}

// Joins the partial results of a block that several shares hold, as the
// absorbed kernel's: blockIdx.x is the share that begins the block,
// blockIdx.y the query tile and an eighth of the 128 elements.  A thread a row,
// four pieces in flight (16 rows of one head on 65536 keys, 152 pieces, 64 us in
// all; two in flight 82; eight 58, but 16 heads x 128 rows on 8192 25.5 for 23.7).
constexpr int kJoinDims = 16;

__global__ void __launch_bounds__(kTile) prefill_join_kernel(const PrefillArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const int4 cut = a.ws_cut[2 * blockIdx.x];
    const int pieces = cut.w;
    if (pieces < 2)
        return;
    constexpr int kParts = kV / kJoinDims;
    const int q = blockIdx.y / kParts, c0 = kJoinDims * (blockIdx.y % kParts), t = threadIdx.x;
    Block k;
    k.b = cut.y;
    block_seq(a, a.cu_q, a.cu_k, k);
    const int row = cut.z * kRows + q * kTile + t;
    if (row >= k.nq)
        return;
    // a share leaves its first segment at 2 p, its last after it
    constexpr int64_t step = 4 * kPartTile;
    const float *rest = a.ws_part + blockIdx.x * step + q * kPartTile;
    const float *first = rest + a.ws_cut[2 * blockIdx.x + 1].x * 2 * kPartTile;
    float top = -INFINITY;
    #pragma unroll 4
    for (int i = 0; i < pieces; ++i)
        top = fmaxf(top, (i == 0 ? first : rest + i * step)[kTile * kV + t]);
    top = top == -INFINITY ? 0.0f : top;
    float acc[kJoinDims] = {}, sum = 0.0f;
    #pragma unroll 4
    for (int i = 0; i < pieces; ++i) {
        const float *f = i == 0 ? first : rest + i * step;
        const float l = f[kTile * kV + kTile + t], w = ex2(f[kTile * kV + t] - top);
        sum = fmaf(w, l, sum);
        #pragma unroll
        for (int e = 0; e < kJoinDims; e += 4) {
            float4 v = *reinterpret_cast<const float4 *>(f + (c0 + e) * kTile + 4 * t);
            if (l == 0.0f)  // no key here: O was not written
                v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            acc[e] = fmaf(w, v.x, acc[e]);
            acc[e + 1] = fmaf(w, v.y, acc[e + 1]);
            acc[e + 2] = fmaf(w, v.z, acc[e + 2]);
            acc[e + 3] = fmaf(w, v.w, acc[e + 3]);
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    __nv_bfloat16 *to = a.out + (int64_t)(k.seq_q + row) * a.ldo_row + cut.x * a.ldo_head + c0;
    #pragma unroll
    for (int e = 0; e < kJoinDims; e += 8) {
        uint32_t v[4];
        #pragma unroll
        for (int x = 0; x < 4; ++x)
            v[x] = pack2(__float_as_uint(acc[e + 2 * x]), __float_as_uint(acc[e + 2 * x + 1]), inv);
        *reinterpret_cast<uint4 *>(to + e) = make_uint4(v[0], v[1], v[2], v[3]);
    }
    if (a.lse && c0 == 0)
        a.lse[(int64_t)(k.seq_q + row) * a.ld_lse + cut.x] =
            sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

inline size_t cut_bytes()
{
    return ((size_t)2 * kMaxShares * sizeof(int4) + 255) / 256 * 256;
}

// bf16 [rows, H, dim] with these strides (elements) as bytes; boxes of 64
// elements of one head of 128 rows.  Strides over one element are free.
inline bool encode_rows(CUtensorMap *map, const uint16_t *p, int dim, int H, int rows, int64_t ld_row,
                 int64_t ld_head)
{
    const uint64_t dims[3] = {(uint64_t)(2 * dim), (uint64_t)H, (uint64_t)rows};
    const uint64_t str[2] = {(uint64_t)(H > 1 ? 2 * ld_head : 2 * dim),
                             (uint64_t)(rows > 1 ? 2 * ld_row : 2 * dim)};
    const uint32_t box[3] = {128, 1, kTile};
    return encode_tma_u8(map, 3, p, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Fills in the rest of a call's arguments and launches it.
template <bool kRope>
idx_status run_prefill(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tr,
                       const CUtensorMap &tv, PrefillArgs &a, void *ws, cudaStream_t stream)
{
    a.uncut = a.Tk <= kUncutKeys;
    a.status = device_status_ptr();
    if (!a.status)
        return IDX_ERR_CUDA;
    a.ws_cut = static_cast<int4 *>(ws);
    a.ws_part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + cut_bytes());
    static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return IDX_ERR_CUDA;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(prefill_kernel<kRope>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Lay<kRope>::kSmem) != cudaSuccess)
            return IDX_ERR_CUDA;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    // few blocks on few keys: no more CTAs than tiles and charges in pairs
    const int64_t blocks = (int64_t)a.Tq / kRows + a.B, tiles = (int64_t)a.Tk / kTile + 1 + kCharge;
    const int most = std::min(sm_count(), kMaxShares);
    const int shares = blocks > most || tiles > 2 * most || a.H > most
                           ? most
                           : (int)std::min<int64_t>(most, std::max<int64_t>(1, blocks * tiles * a.H / 2));
    cudaError_t e = launch_pdl(prefill_kernel<kRope>, dim3(shares), dim3(kThreads),
                               Lay<kRope>::kSmem, stream, tq, tk, tr, tv, a);
    if (e == cudaSuccess && shares > 1 && !a.uncut)
        e = launch_pdl(prefill_join_kernel, dim3(shares - 1, 2 * kV / kJoinDims), dim3(kTile), 0,
                       stream, a);
    return launch_status(e);
}

// Device scratch of a call.
inline size_t prefill_workspace(int Tq, int Tk, int H)
{
    if (Tq <= 0 || H <= 0 || Tk <= kUncutKeys)
        return 0;
    return cut_bytes() + (size_t)2 * kMaxShares * 2 * kPartTile * sizeof(float);
}

} // namespace
} // namespace idx
