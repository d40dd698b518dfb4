// idx_internal.h -- host-side helpers shared by the library's translation
// units (not part of the public ABI).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/idx.h"
#include <nvtx3/nvToolsExt.h>

namespace idx {

// Device address of the sticky status word of the current device.
unsigned int *device_status_ptr();

// Number of SMs of the current device (cached per device).
int sm_count();

// 16-byte alignment check of a device pointer.
inline bool aligned16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// Elements [n0][n1][inner] of `size` bytes, strides in elements.
struct Strided {
    const void *p;
    int64_t n0, s0, n1, s1, inner;
    int size;
};

// Whether its elements lie apart, as those of a written tensor have to: one outer
// dimension's steps pass over all that the other one covers.
inline bool lie_apart(const Strided &t)
{
    using Wide = __int128;  // counts and strides are the caller's
    const bool swap = t.n0 > 1 && t.n1 > 1 && t.s0 < t.s1;
    const int64_t no = swap ? t.n1 : t.n0, so = swap ? t.s1 : t.s0;  // the outer one
    const int64_t ni = swap ? t.n0 : t.n1, si = swap ? t.s0 : t.s1;
    if (ni > 1 && si < t.inner)
        return false;
    return no <= 1 || so >= (ni > 1 ? (Wide)si * (ni - 1) : 0) + t.inner;
}

// Whether bytes [p, p + n) and [q, q + m) meet (nothing meets none).
inline bool meet(const void *p, __int128 n, const void *q, __int128 m)
{
    const __int128 a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && n > 0 && m > 0 && a < b + m && b < a + n;
}

// Bytes from the first element to the last one's end.
inline __int128 span(const Strided &t)
{
    return t.n0 <= 0 || t.n1 <= 0 || t.inner <= 0
               ? 0
               : ((__int128)(t.n0 - 1) * t.s0 + (__int128)(t.n1 - 1) * t.s1 + t.inner) * t.size;
}

// Whether two tensors of one shape have no element in common: spans that do not meet,
// or views of the same strides whose elements lie beside one another.
inline bool lie_apart(const Strided &x, const Strided &y)
{
    if (!meet(x.p, span(x), y.p, span(y)))
        return true;
    if ((x.n0 > 1 && x.s0 != y.s0) || (x.n1 > 1 && x.s1 != y.s1) || !lie_apart(x))
        return false;
    // The spans meet, so their distance is in range.  An element of both is i outer steps, j
    // inner ones and k elements away; what is left after the outer steps is under one of them.
    const int64_t bytes = (int64_t)(reinterpret_cast<uintptr_t>(y.p) - reinterpret_cast<uintptr_t>(x.p));
    if (bytes % x.size != 0)
        return false;
    const auto floor_of = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
    const bool swap = x.n0 > 1 && x.n1 > 1 && x.s0 < x.s1;
    const int64_t no = swap ? x.n1 : x.n0, so = swap ? x.s1 : x.s0;
    const int64_t ni = swap ? x.n0 : x.n1, si = swap ? x.s0 : x.s1;
    const int64_t d = bytes / x.size, i0 = no > 1 ? floor_of(d, so) : 0;
    for (int64_t i = i0; i <= i0 + (no > 1); ++i) {
        const int64_t r = d - (no > 1 ? i * so : 0), j0 = ni > 1 ? floor_of(r, si) : 0;
        for (int64_t j = j0; j <= j0 + (ni > 1); ++j) {
            const int64_t k = r - (ni > 1 ? j * si : 0);
            if (i > -no && i < no && j > -ni && j < ni && k > -x.inner && k < x.inner)
                return false;
        }
    }
    return true;
}

// Encode a tiled TMA descriptor of uint8 elements (rank 2 or 3).  Returns
// false if the driver rejects the arguments.
bool encode_tma_u8(CUtensorMap *map, int rank, const void *base, const uint64_t *dims,
                   const uint64_t *strides_bytes, const uint32_t *box, CUtensorMapSwizzle swz);

// Chunked top-k pieces (idx_select.cu) for a logits call that computes the
// top-k's digit-1 histograms itself: the plan kernel (with zero_cvalid it
// also clears the per-chunk valid counts), the phases (hist_done: start at
// the filter), where the counts live in ws, and whether idx_topk would take
// the chunked path for these arguments.
idx_status topk_chunked_plan(const int32_t *lengths, int64_t ld, int rows, void *ws,
                             int zero_cvalid, cudaStream_t s);
idx_status topk_chunked_phases(const float *logits, int64_t ld, int rows, const int32_t *lengths,
                               int k, int32_t *out, int64_t ld_out, void *ws, int vec_ok,
                               int hist_done, cudaStream_t s);
int topk_chunked_counts(void *ws, int rows, int64_t ld, uint32_t **hist, uint32_t **valid,
                        uint32_t **cvalid);
bool topk_takes_chunked(const float *logits, int64_t ld, int rows, int k, const void *ws,
                        size_t ws_bytes);

// An NVTX range around one C-ABI call, named after the entry point, so a
// profiler's timeline shows which call launched which kernels.  NVTX is
// header-only: without a profiler attached a range costs a test of one
// function pointer.
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};
#define IDX_NVTX_RANGE(name) ::idx::NvtxRange idx_nvtx_range_(name)

inline idx_status launch_status(cudaError_t e)
{
    return e == cudaSuccess ? IDX_OK : IDX_ERR_CUDA;
}

// Launch with programmatic stream serialization: the kernel may begin while
// the previous kernel on the stream finishes; it must call pdl_wait() before
// touching memory an earlier kernel may use.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

} // namespace idx
