// idx_latent.cuh -- the latent cache's layout and the bounds-checked look-ups
// shared by its writer, its read-back and the attention kernels.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "idx_common.cuh"
#include "idx_internal.h"

namespace idx {

constexpr int kLatent = 512;                 // latent elements of a token (key and value)
constexpr int kLatRope = 64;                 // rotated elements of a token (key only)
constexpr int kLatTok = kLatent + kLatRope;  // 576
constexpr int kLatGroup = 64;                // latents under one e8m0 scale
constexpr int kLatGroups = kLatent / kLatGroup;
constexpr int kLatFp8TokBytes = kLatent + 2 * kLatRope + kLatGroups;
constexpr int kLatBf16TokBytes = 2 * kLatTok;

// The pool of pages as the kernels get it.
struct LatentPool {
    const uint8_t *base;
    int64_t stride;  // bytes between pages
    int num_pages;
    int page_size;
    // slot / page_size = __umulhi(slot, magic) >> shift for slots below 2^31
    // (magic = 0: page_size is 1)
    uint32_t magic;
    int shift;
};

inline LatentPool make_pool(const uint8_t *base, int64_t stride, int num_pages, int page_size)
{
    // rounding up: with l = ceil(log2 d), m = floor(2^(31 + l) / d) + 1 is below
    // 2^32 and n m / 2^(31 + l) exceeds n / d by less than 1 / d for n < 2^31
    LatentPool p = {base, stride, num_pages, page_size, 0, 0};
    if (page_size > 1) {
        int l = 1;
        while ((1ll << l) < page_size)
            ++l;
        p.magic = (uint32_t)((1ull << (31 + l)) / (uint64_t)page_size + 1);
        p.shift = l - 1;
    }
    return p;
}

// Host check of a pool: 0 good, otherwise the status to return.
inline idx_status check_pool(const uint8_t *base, int64_t stride, int num_pages, int page_size,
                             idx_latent_format fmt)
{
    if (page_size <= 0 || num_pages < 0 || (fmt != IDX_LATENT_BF16 && fmt != IDX_LATENT_FP8_E4M3))
        return IDX_ERR_INVALID_ARG;
    const int64_t tok = fmt == IDX_LATENT_BF16 ? kLatBf16TokBytes : kLatFp8TokBytes;
    if (!base || stride < page_size * tok)
        return IDX_ERR_INVALID_ARG;
    // slots are int32: the last one has to be
    if ((int64_t)num_pages * page_size > INT32_MAX || !aligned16(base) || stride % 16 != 0)
        return IDX_ERR_UNSUPPORTED;
    return IDX_OK;
}

// Page of a slot (or of a token within its sequence), below 2^31.
IDX_DEVFN int page_of(const LatentPool &p, int slot)
{
    return p.magic ? (int)(__umulhi((uint32_t)slot, p.magic) >> p.shift) : slot;
}

} // namespace idx
