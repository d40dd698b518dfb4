// idx_grouped_prefill.cu -- attention of whole prompts with grouped heads, several
// query heads to a key head: its entry points.  The kernels are idx_prefill.cuh's.
#include "idx_prefill.cuh"

using namespace idx;

extern "C" size_t idx_grouped_prefill_workspace_size(int Tq, int Tk, int H)
{
    return prefill_workspace(Tq, Tk, H);
}

extern "C" idx_status idx_grouped_prefill(const uint16_t *q, int64_t ldq_row, int64_t ldq_head,
                                          const uint16_t *k, int64_t ldk_row, int64_t ldk_head,
                                          const uint16_t *v, int64_t ldv_row, int64_t ldv_head,
                                          const int32_t *cu_q, const int32_t *cu_k, int B, int Tq,
                                          int Tk, int H, int kv_heads, int D, float scale,
                                          int causal, uint16_t *out, int64_t ldo_row,
                                          int64_t ldo_head, float *lse, int64_t ld_lse, void *ws,
                                          size_t ws_bytes, idx_stream_t stream)
{
    IDX_NVTX_RANGE("idx_grouped_prefill");
    if (B < 0 || Tq < 0 || Tk < 0 || H <= 0 || kv_heads <= 0 || D <= 0)
        return IDX_ERR_INVALID_ARG;
    if (B == 0 || Tq == 0)
        return IDX_OK;
    if (!q || !cu_q || !cu_k || !out || (Tk > 0 && (!k || !v)) || !(scale > 0.0f) ||
        !(scale * kLog2e <= 3.4e38f) || ldq_head < D || ldq_row < 0 || ldk_head < D ||
        ldk_row < 0 || ldv_head < D || ldv_row < 0 || ldo_head < D || ldo_row < 0 ||
        (lse && ld_lse < H))
        return IDX_ERR_INVALID_ARG;
    if (D != kV || H > 65535 || H % kv_heads != 0 || !aligned16(q) || !aligned16(k) ||
        !aligned16(v) || !aligned16(out) ||
        (ldq_row | ldq_head | ldk_row | ldk_head | ldv_row | ldv_head | ldo_row | ldo_head) % 8 != 0)
        return IDX_ERR_UNSUPPORTED;
    const size_t need = idx_grouped_prefill_workspace_size(Tq, Tk, H);
    if (need > 0 && (!ws || !aligned16(ws) || ws_bytes < need))
        return IDX_ERR_WORKSPACE;
    if (Tq > INT32_MAX - 2 * kRows || Tk > INT32_MAX - 2 * kTile)
        return IDX_ERR_UNSUPPORTED;  // rows and tiles are counted past the end
    if (!lie_apart({out, Tq, ldo_row, H, ldo_head, D, 2}))
        return IDX_ERR_INVALID_ARG;
    CUtensorMap tq, tk, tv;
    if (!encode_rows(&tq, q, kV, H, Tq, ldq_row, ldq_head))
        return IDX_ERR_UNSUPPORTED;
    if (Tk > 0) {
        if (!encode_rows(&tk, k, kV, kv_heads, Tk, ldk_row, ldk_head) ||
            !encode_rows(&tv, v, kV, kv_heads, Tk, ldv_row, ldv_head))
            return IDX_ERR_UNSUPPORTED;
    } else {
        tk = tv = tq;  // no key tile is read
    }
    PrefillArgs a = {};
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.B = B;
    a.Tq = Tq;
    a.Tk = Tk;
    a.H = H;
    a.group = H / kv_heads;
    a.scale_log2 = scale * kLog2e;
    a.causal = causal;
    a.out = reinterpret_cast<__nv_bfloat16 *>(out);
    a.ldo_row = ldo_row;
    a.ldo_head = ldo_head;
    a.lse = lse;
    a.ld_lse = ld_lse;
    return run_prefill<false>(tq, tk, tk, tv, a, ws, (cudaStream_t)stream);
}
