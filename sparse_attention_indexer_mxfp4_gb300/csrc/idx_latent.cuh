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
    int page_shift;  // log2(page_size), or -1
};

inline LatentPool make_pool(const uint8_t *base, int64_t stride, int num_pages, int page_size)
{
    LatentPool p = {base, stride, num_pages, page_size, -1};
    for (int s = 0; s < 31; ++s)
        if (page_size == 1 << s)
            p.page_shift = s;
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

// Slot -> page and offset; false for a slot outside the pool.
IDX_DEVFN bool slot_place(const LatentPool &p, int64_t slot, int64_t *page_byte, int *off)
{
    if (slot < 0)
        return false;
    int64_t page;
    if (p.page_shift >= 0) {
        page = slot >> p.page_shift;
        *off = (int)(slot & (p.page_size - 1));
    } else {
        page = slot / p.page_size;
        *off = (int)(slot - page * p.page_size);
    }
    *page_byte = page * p.stride;
    return page < p.num_pages;
}

IDX_DEVFN int page_of(const LatentPool &p, int t)
{
    return p.page_shift >= 0 ? t >> p.page_shift : t / p.page_size;
}

} // namespace idx
