// idx_latent_prefill.cu -- expanded latent attention of ragged sequences:
// s = scale * (q[:128] . k + q[128:] . k_rope), out = softmax(s) . v.
//
// A CTA takes up to two tiles of 128 queries of one head and walks the keys
// they see, 128 at a time, with a running maximum and sum:
//
//     S [128 queries x 128 keys] = Q [128 x 192] . K^T   (12 MMAs, 128 x 128 x 16)
//     O [128 x 128]             += P [128 x 128] . V     (2 x 8 MMAs, 128 x 64 x 16)
//
// The two tiles take turns: while the softmax warps of one work, the tensor
// cores do the other's products, and both read each key tile once.  Scores,
// weights and sums stay in tensor memory: S (128 columns) is overwritten by P
// in bf16, which the second product takes as its A operand from there.  The
// tensor cores bound it: 1280 cycles a tile pair against 1024 of exponentials.
//
// Keys and values come by TMA in pieces of 64 elements of 128 tokens (16 KB,
// 128-byte swizzled), five a tile (three of K, the last shared by all heads,
// two of V), through a ring of eight: K^T is read K-major, V M-major, as they
// lie.  The running maximum is only raised when a score exceeds it by 2^40
// (32-bit sums lose nothing by that), so rescaling O is rare after a row's
// first tile.
//
// Warps: 0-3 and 4-7 softmax of the two tiles, a thread a query; 8 issues TMA;
// 9 issues the products.
#include <atomic>
#include <cuda_bf16.h>

#include "idx_common.cuh"
#include "idx_internal.h"

namespace idx {
namespace {

constexpr int kNope = 128, kRope = 64, kV = 128, kQk = kNope + kRope;
constexpr int kTile = 128;                      // queries and keys of a tile
constexpr int kPiece = kTile * 128;             // bytes of 64 elements of a tile's tokens
constexpr int kQPieces = kQk / 64, kVPieces = kV / 64, kPieces = kQPieces + kVPieces;
constexpr int kRing = 8;
constexpr int kWarpLoad = 8, kWarpMma = 9;
constexpr int kThreads = 320;
constexpr int kOffRing = 2 * kQPieces * kPiece;
constexpr int kOffBar = kOffRing + kRing * kPiece;
constexpr int kBars = 2 * kRing + 9;
constexpr int kOffMisc = kOffBar + 8 * kBars;  // tmem base, abort flag
constexpr int kSmem = kOffMisc + 16 + 1024;    // the base is aligned to 1024 in the kernel
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
constexpr uint32_t kColS = 0, kColO = 256;     // tensor memory columns, 128 a query tile
constexpr float kLazy = 40.0f;                 // a score may exceed its running maximum by 2^40
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

struct PrefillArgs {
    const int32_t *cu_q, *cu_k;
    int B, Tq, Tk, H;
    int tiles;  // query tiles of a CTA (1 or 2)
    float scale_log2;
    int causal;
    __nv_bfloat16 *out;
    int64_t ldo_row, ldo_head;
    float *lse;
    int64_t ld_lse;
    unsigned int *status;
};

// A CTA's queries: rows q0 .. of a sequence of nq queries and nk keys.
struct Block {
    int seq_q, seq_k, nq, nk, q0;
};

// Finds block t of all sequences' blocks of `rows` queries, the last of a
// sequence first (causal: they see the most keys).  One warp; false past the end.
__device__ __forceinline__ bool find_block(const PrefillArgs &a, int t, int rows, Block &k)
{
    const int lane = lane_id();
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        int lo = 0, n = 0;
        if (b < a.B) {
            lo = min(max(a.cu_q[b], 0), a.Tq);
            n = max(0, min(a.cu_q[b + 1], a.Tq) - lo);
        }
        const int blocks = (n + rows - 1) / rows;
        int upto = blocks;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? v : 0;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, upto > t);
        if (past) {
            const int src = __ffs(past) - 1;
            const int first = __shfl_sync(0xffffffffu, upto - blocks, src);
            const int count = __shfl_sync(0xffffffffu, blocks, src);
            k.seq_q = __shfl_sync(0xffffffffu, lo, src);
            k.nq = __shfl_sync(0xffffffffu, n, src);
            k.q0 = (count - 1 - (t - first)) * rows;
            k.seq_k = min(max(a.cu_k[b0 + src], 0), a.Tk);
            k.nk = max(0, min(a.cu_k[b0 + src + 1], a.Tk) - k.seq_k);
            return true;
        }
        t -= __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}

// Keys that query row i of the sequence sees.
__device__ __forceinline__ int keys_seen(const PrefillArgs &a, const Block &k, int i)
{
    return a.causal ? min(k.nk, max(0, i + k.nk - k.nq + 1)) : k.nk;
}

// Key tiles of query tile q of the block (0: it has no queries, or they no keys).
__device__ __forceinline__ int key_tiles(const PrefillArgs &a, const Block &k, int q)
{
    const int first = k.q0 + q * kTile, last = min(first + kTile, k.nq) - 1;
    if (q >= a.tiles || last < first)
        return 0;
    return (keys_seen(a, k, last) + kTile - 1) / kTile;
}

__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_r,
                          const __grid_constant__ CUtensorMap tm_v, const PrefillArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *full = bar, *empty = bar + kRing;
    uint64_t *s_full = bar + 2 * kRing, *p_full = s_full + 2, *pv_done = s_full + 4;
    uint64_t *q_full = s_full + 6, *tail = s_full + 7, *drain = s_full + 8;
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int head = blockIdx.y;

    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(tail, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(misc, 512);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_launch_dependents();
    Block k;
    const bool some = find_block(a, blockIdx.x, a.tiles * kTile, k);
    // key tiles of the two query tiles
    const int nt0 = some ? key_tiles(a, k, 0) : 0, nt1 = some ? key_tiles(a, k, 1) : 0;
    const int most = max(nt0, nt1);
    __syncthreads();
    tc_fence_after();
    // one value for the warp, as the compiler sees it too
    const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);

    if (!some) {
        // nothing here: only the tensor memory to give back
    } else if (warp < kWarpLoad) {
        // ------------------------------------------------ softmax, epilogue
        const int q = warp >> 2;
        const int row = k.q0 + q * kTile + (tid & 127);
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t col_s = tmem + lanes + kColS + q * 128, col_o = tmem + lanes + kColO + q * 128;
        const float sl = a.scale_log2;
        // rows past the sequence's queries take part with no key
        const int seen = row < k.nq ? keys_seen(a, k, row) : 0;
        const int seen_first = __shfl_sync(0xffffffffu, seen, 0);  // the warp's fewest, if it has them
        const bool whole_warp = __all_sync(0xffffffffu, row < k.nq);
        const int nt = q ? nt1 : nt0;
        float m = -INFINITY, l = 0.0f;
        for (int j = 0; j < nt; ++j) {
            // after an abort the waits return at once and the loop runs out
            (void)mbar_wait(&s_full[q], j & 1, abort_flag, a.status);
            __syncwarp();
            tc_fence_after();
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
                if (j > 0) {
                    (void)mbar_wait(&pv_done[q], (j - 1) & 1, abort_flag, a.status);
                    __syncwarp();
                    tc_fence_after();
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
            float sum[4] = {};
            #pragma unroll
            for (int c = 0; c < 2; ++c) {
                // weights as bf16 (half a step of 2^-8 each), two a column
                uint32_t w[32];
                #pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const int at = 2 * e & 31;
                    const float x = ex2(fmaf(__uint_as_float(r[2 * c + (e >> 4)][at]), sl, nm));
                    const float y = ex2(fmaf(__uint_as_float(r[2 * c + (e >> 4)][at + 1]), sl, nm));
                    sum[e & 3] += x + y;
                    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
                    w[e] = *reinterpret_cast<const uint32_t *>(&v);
                }
                tmem_st_32x32b_x32(col_s + 32 * c, w);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&p_full[q]);
        }
        if (nt > 0) {
            (void)mbar_wait(&pv_done[q], (nt - 1) & 1, abort_flag, a.status);
            __syncwarp();
            tc_fence_after();
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const bool mine = q < a.tiles && row < k.nq;
        __nv_bfloat16 *to = a.out + (int64_t)(k.seq_q + row) * a.ldo_row + head * a.ldo_head;
        #pragma unroll 1
        for (int c = 0; c < 128; c += 16) {
            uint32_t o[16];
            if (nt > 0) {
                tmem_ld_32x32b_x16(col_o + c, o);
                tmem_ld_wait();
            } else {
                #pragma unroll
                for (int e = 0; e < 16; ++e)
                    o[e] = 0;
            }
            uint32_t w[8];
            #pragma unroll
            for (int e = 0; e < 8; ++e) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[2 * e]) * inv,
                                                               __uint_as_float(o[2 * e + 1]) * inv);
                w[e] = *reinterpret_cast<const uint32_t *>(&v);
            }
            if (mine) {
                *reinterpret_cast<uint4 *>(to + c) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4 *>(to + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
        if (mine && a.lse)
            a.lse[(int64_t)(k.seq_q + row) * a.ld_lse + head] =
                l == 0.0f ? -INFINITY : ((m == -INFINITY ? 0.0f : m) + log2f(l)) * kLn2;
        tc_fence_before();
    } else if (warp == kWarpLoad) {
        // ------------------------------------------------------------- TMA
        const bool one = elect_one();
        int n = 0;           // pieces issued
        bool q_flying = false, ok = most > 0;
        if (ok && one) {
            mbar_arrive_expect_tx(q_full, (nt1 > 0 ? 2 : 1) * kQPieces * kPiece);
            #pragma unroll 1
            for (int q = 0; q < (nt1 > 0 ? 2 : 1); ++q) {
                #pragma unroll 1
                for (int c = 0; c < kQPieces; ++c)
                    tma_load_3d(smem + (q * kQPieces + c) * kPiece, &tm_q, q_full, 128 * c, head,
                                k.seq_q + k.q0 + q * kTile);
            }
        }
        q_flying = ok;
        bool tail_flying = false;
        for (int j = 0; ok && j < most; ++j) {
            const int t0 = k.seq_k + j * kTile, rem = k.nk - j * kTile;
            #pragma unroll 1
            for (int c = 0; c < kPieces; ++c, ++n) {
                const int slot = n & (kRing - 1);
                if (n >= kRing) {
                    ok = mbar_wait(&empty[slot], ((n >> 3) - 1) & 1, abort_flag, a.status);
                    if (!ok)
                        break;
                }
                __syncwarp();
                uint8_t *to = smem + kOffRing + slot * kPiece;
                const bool cut = c >= kQPieces && rem < kTile;  // values past the sequence
                if (one) {
                    uint64_t *b = cut ? tail : &full[slot];
                    mbar_arrive_expect_tx(b, kPiece);
                    if (c < 2)
                        tma_load_3d(to, &tm_k, b, 128 * c, head, t0);
                    else if (c == 2)
                        tma_load_2d(to, &tm_r, b, 0, t0);
                    else
                        tma_load_3d(to, &tm_v, b, 128 * (c - kQPieces), head, t0);
                }
                __syncwarp();
                if (cut) {
                    // a weight of zero does not hide what is not finite:
                    // another sequence's values become zeros here
                    tail_flying = true;
                    ok = mbar_wait(tail, c - kQPieces, abort_flag, a.status);
                    if (!ok)
                        break;
                    tail_flying = false;
                    for (int e = rem * 8 + lane; e < kTile * 8; e += 32)
                        st_shared_v4(smem_u32(to) + 16 * e, 0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&full[slot]);
                }
            }
        }
        if (*abort_flag) {
            // the copies in flight land before the CTA leaves
            if (q_flying)
                (void)mbar_wait_drain(q_full, 0);
            if (tail_flying)
                (void)mbar_wait_drain(tail, 0);
            for (int i = n > kRing ? n - kRing : 0; i < n; ++i)
                (void)mbar_wait_drain(&full[i & (kRing - 1)], (i >> 3) & 1);
        }
    } else {
        // ------------------------------------------------------------ MMAs
        const bool one = elect_one();
        const uint32_t id_s = idesc_bf16(kTile, kTile, false, false);
        const uint32_t id_v = idesc_bf16(kTile, 64, false, true);
        bool ok = most > 0 && mbar_wait(q_full, 0, abort_flag, a.status);
        // S of query tile q and key tile j; the last query tile frees the keys
        const auto scores = [&](int q, int j) {
            const bool last = q == 1 || nt1 <= j;
            const uint32_t qd = desc_lo(sbase + q * kQPieces * kPiece);
            #pragma unroll
            for (int c = 0; c < kQPieces; ++c) {
                const int n = j * kPieces + c, slot = n & (kRing - 1);
                if (!mbar_wait(&full[slot], (n >> 3) & 1, abort_flag, a.status))
                    return false;
                __syncwarp();
                tc_fence_after();
                const uint32_t kd = desc_lo(sbase + kOffRing + slot * kPiece);
                #pragma unroll
                for (int e = 0; e < 4; ++e)
                    mma_f16(tmem + kColS + q * 128, qd + (c * kPiece >> 4) + 2 * e, kd + 2 * e,
                            kDescHiSw128, id_s, c + e > 0 ? 1u : 0u, one);
                mma_commit_if(&empty[slot], one && last);
            }
            mma_commit_if(&s_full[q], one);
            return true;
        };
        const auto values = [&](int q, int j) {
            const bool last = q == 1 || nt1 <= j;
            if (!mbar_wait(&p_full[q], j & 1, abort_flag, a.status))
                return false;
            #pragma unroll
            for (int c = 0; c < kVPieces; ++c) {
                const int n = j * kPieces + kQPieces + c, slot = n & (kRing - 1);
                if (!mbar_wait(&full[slot], (n >> 3) & 1, abort_flag, a.status))
                    return false;
                __syncwarp();
                tc_fence_after();
                const uint32_t vd = desc_lo(sbase + kOffRing + slot * kPiece);
                #pragma unroll
                for (int e = 0; e < 8; ++e)
                    mma_f16_ts(tmem + kColO + q * 128 + 64 * c, tmem + kColS + q * 128 + 8 * e,
                               vd + e * (2048 >> 4), kDescHiSw128, id_v, j + e > 0 ? 1u : 0u, one);
                mma_commit_if(&empty[slot], one && last);
            }
            mma_commit_if(&pv_done[q], one);
            return true;
        };
        if (ok && nt0 > 0)
            ok = scores(0, 0);
        if (ok && nt1 > 0)
            ok = scores(1, 0);
        for (int j = 0; ok && j < most; ++j) {
            #pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int nt = q ? nt1 : nt0;
                if (ok && j < nt)
                    ok = values(q, j);
                if (ok && j + 1 < nt)
                    ok = scores(q, j + 1);
            }
        }
        if (*abort_flag) {
            if (one)
                mma_commit(drain);
            __syncwarp();
            (void)mbar_wait_drain(drain, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma)
        tmem_dealloc(tmem, 512);
}

// bf16 [rows, H, dim] with these strides (elements) as bytes; boxes of 64
// elements of one head of 128 rows.  Strides over one element are free.
bool encode_rows(CUtensorMap *map, const uint16_t *p, int dim, int H, int rows, int64_t ld_row,
                 int64_t ld_head)
{
    const uint64_t dims[3] = {(uint64_t)(2 * dim), (uint64_t)H, (uint64_t)rows};
    const uint64_t str[2] = {(uint64_t)(H > 1 ? 2 * ld_head : 2 * dim),
                             (uint64_t)(rows > 1 ? 2 * ld_row : 2 * dim)};
    const uint32_t box[3] = {128, 1, kTile};
    return encode_tma_u8(map, 3, p, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
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
    CUtensorMap tq, tk, tr, tv;
    const uint64_t rdims[2] = {2 * kRope, (uint64_t)Tk};
    const uint64_t rstr[1] = {(uint64_t)(Tk > 1 ? 2 * ld_rope : 2 * kRope)};
    const uint32_t rbox[2] = {128, kTile};
    if (!encode_rows(&tq, q, kQk, H, Tq, ldq_row, ldq_head))
        return IDX_ERR_UNSUPPORTED;
    if (Tk > 0) {
        if (!encode_rows(&tk, k, kNope, H, Tk, ldk_row, ldk_head) ||
            !encode_rows(&tv, v, kV, H, Tk, ldv_row, ldv_head) ||
            !encode_tma_u8(&tr, 2, k_rope, rdims, rstr, rbox, CU_TENSOR_MAP_SWIZZLE_128B))
            return IDX_ERR_UNSUPPORTED;
    } else {
        tk = tr = tv = tq;  // no key tile is read
    }
    PrefillArgs a = {};
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.B = B;
    a.Tq = Tq;
    a.Tk = Tk;
    a.H = H;
    a.scale_log2 = scale * kLog2e;
    a.causal = causal;
    a.out = reinterpret_cast<__nv_bfloat16 *>(out);
    a.ldo_row = ldo_row;
    a.ldo_head = ldo_head;
    a.lse = lse;
    a.ld_lse = ld_lse;
    a.status = device_status_ptr();
    if (!a.status)
        return IDX_ERR_CUDA;
    // two query tiles a CTA unless that leaves SMs without one
    a.tiles = (int64_t)(Tq / (2 * kTile)) * H >= sm_count() ? 2 : 1;
    static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return IDX_ERR_CUDA;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(latent_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmem) != cudaSuccess)
            return IDX_ERR_CUDA;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    // every sequence ends in at most one block that is not full
    const int64_t blocks = (int64_t)Tq / (a.tiles * kTile) + B;
    if (blocks > INT32_MAX)
        return IDX_ERR_UNSUPPORTED;
    return launch_status(launch_pdl(latent_prefill_kernel, dim3((unsigned)blocks, H),
                                    dim3(kThreads), kSmem, (cudaStream_t)stream, tq, tk, tr, tv,
                                    a));
}
