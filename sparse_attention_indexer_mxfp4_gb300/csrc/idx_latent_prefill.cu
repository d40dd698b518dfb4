// idx_latent_prefill.cu -- the expanded form of latent attention: its entry
// points.  The kernels are idx_prefill.cuh's.
#include "idx_prefill.cuh"

using namespace idx;

namespace {

constexpr int kNope = 128, kRope = 64, kQk = kNope + kRope;

} // namespace

extern "C" size_t idx_latent_prefill_workspace_size(int Tq, int Tk, int H)
{
    return prefill_workspace(Tq, Tk, H);
}

extern "C" idx_status idx_latent_prefill(const uint16_t *q, int64_t ldq_row, int64_t ldq_head,
                                         const uint16_t *k, int64_t ldk_row, int64_t ldk_head,
                                         const uint16_t *k_rope, int64_t ld_rope,
                                         const uint16_t *v, int64_t ldv_row, int64_t ldv_head,
                                         const int32_t *cu_q, const int32_t *cu_k, int B, int Tq,
                                         int Tk, int H, int d_nope, int d_rope, int d_v,
                                         float scale, int causal, uint16_t *out, int64_t ldo_row,
                                         int64_t ldo_head, float *lse, int64_t ld_lse, void *ws,
                                         size_t ws_bytes, idx_stream_t stream)
{
    IDX_NVTX_RANGE("idx_latent_prefill");
    if (B < 0 || Tq < 0 || Tk < 0 || H <= 0 || d_nope <= 0 || d_rope < 0 || d_v <= 0)
        return IDX_ERR_INVALID_ARG;
    if (B == 0 || Tq == 0)
        return IDX_OK;
    if (!q || !cu_q || !cu_k || !out || (Tk > 0 && (!k || !k_rope || !v)) || !(scale > 0.0f) ||
        !(scale * kLog2e <= 3.4e38f) || ldq_head < (int64_t)d_nope + d_rope || ldq_row < 0 ||
        ldk_head < d_nope || ldk_row < 0 || ld_rope < d_rope || ldv_head < d_v || ldv_row < 0 ||
        ldo_head < d_v || ldo_row < 0 || (lse && ld_lse < H))
        return IDX_ERR_INVALID_ARG;
    if (d_nope != kNope || d_rope != kRope || d_v != kV || H > 65535 || !aligned16(q) ||
        !aligned16(k) || !aligned16(k_rope) || !aligned16(v) || !aligned16(out) ||
        (ldq_row | ldq_head | ldk_row | ldk_head | ld_rope | ldv_row | ldv_head | ldo_row |
         ldo_head) % 8 != 0)
        return IDX_ERR_UNSUPPORTED;
    const size_t need = idx_latent_prefill_workspace_size(Tq, Tk, H);
    if (need > 0 && (!ws || !aligned16(ws) || ws_bytes < need))
        return IDX_ERR_WORKSPACE;
    if (Tq > INT32_MAX - 2 * kRows || Tk > INT32_MAX - 2 * kTile)
        return IDX_ERR_UNSUPPORTED;  // rows and tiles are counted past the end
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
    a.group = 1;
    a.scale_log2 = scale * kLog2e;
    a.causal = causal;
    a.out = reinterpret_cast<__nv_bfloat16 *>(out);
    a.ldo_row = ldo_row;
    a.ldo_head = ldo_head;
    a.lse = lse;
    a.ld_lse = ld_lse;
    return run_prefill<true>(tq, tk, tr, tv, a, ws, (cudaStream_t)stream);
}
