// idx_kv4.cuh -- the 4-bit key and value cache of grouped heads: its layout,
// the look-ups and the conversions that its writer, its read-back, the
// attention and the eviction share.
//
// A token of one key head is 128 key and 128 value elements in e2m1 with one
// e8m0 scale for each 32.  Block-flat pages: the codes of all keys, of all
// values (64 bytes a token), the scales of the keys, of the values (4 bytes a
// token), each [key heads][page_size].
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "idx_common.cuh"
#include "idx_internal.h"
#include "idx_latent.cuh"

namespace idx {

constexpr int kKv4Dim = 128;
constexpr int kKv4Codes = kKv4Dim / 2;    // bytes of a token's keys or values
constexpr int kKv4Groups = kKv4Dim / 32;  // scales of them, a byte each
constexpr int kKv4TokBytes = 2 * (kKv4Codes + kKv4Groups);

// Where a page's parts begin.
struct Kv4Pool {
    LatentPool p;
    int heads;
    int64_t side;    // codes of the keys: the values' follow
    int64_t scales;  // where the keys' scales begin
    int64_t scale_side;
};

inline Kv4Pool make_kv4_pool(const uint8_t *base, int64_t stride, int num_pages, int page_size,
                             int heads)
{
    const int64_t n = (int64_t)page_size * heads;
    return {make_pool(base, stride, num_pages, page_size), heads, n * kKv4Codes,
            2 * n * kKv4Codes, n * kKv4Groups};
}

// Host check of a pool: 0 good, otherwise the status to return.
inline idx_status check_kv4_pool(const uint8_t *base, int64_t stride, int num_pages, int page_size,
                                 int heads)
{
    if (page_size <= 0 || num_pages < 0 || heads <= 0 || !base)
        return IDX_ERR_INVALID_ARG;
    // (64-bit products of two ints and 136 stay in range)
    if ((int64_t)page_size * heads > INT64_MAX / (2 * kKv4TokBytes) ||
        stride < (int64_t)page_size * heads * kKv4TokBytes)
        return IDX_ERR_INVALID_ARG;
    // slots are int32, and so are places within a page
    if ((int64_t)num_pages * page_size > INT32_MAX || !aligned16(base) || stride % 16 != 0 ||
        stride > INT32_MAX)
        return IDX_ERR_UNSUPPORTED;
    return IDX_OK;
}

// Byte of the key codes of a head's token; the values' are `side` further.
IDX_DEVFN int64_t kv4_codes_at(const Kv4Pool &c, int page, int head, int off)
{
    return page * c.p.stride + ((int64_t)head * c.p.page_size + off) * kKv4Codes;
}

// Byte of the key scales; the values' are `scale_side` further.
IDX_DEVFN int64_t kv4_scales_at(const Kv4Pool &c, int page, int head, int off)
{
    return page * c.p.stride + c.scales + ((int64_t)head * c.p.page_size + off) * kKv4Groups;
}

// The eight e2m1 codes of a word as four pairs of f16, which hold them exactly
// (element 2 i is the low nibble of byte i).
IDX_DEVFN void e2m1_to_f16x2(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// The four scales of a word, 2^(byte - 127) (255: NaN).
IDX_DEVFN void e8m0_to_float(uint32_t w, float (&s)[4])
{
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %0, a;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    s[0] = __uint_as_float(lo << 16);
    s[1] = __uint_as_float(lo & 0xffff0000u);
    s[2] = __uint_as_float(hi << 16);
    s[3] = __uint_as_float(hi & 0xffff0000u);
}

} // namespace idx
