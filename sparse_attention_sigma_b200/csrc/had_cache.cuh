// had_cache.cuh -- the decoder cache of binarized attention: layout, and the
// kernels that write tokens into it and read them back.
//
// A pool holds `pages` pages; a page holds `page` consecutive tokens of one
// sequence (a power of two) for each of `heads` key-value heads.  Of a token
// and head it keeps
//   kbits   d/32 uint32   the signs of the key (bit 1: sign -1), exact;
//   vcodes  d/2 bytes     the value in 4 bits, element 2i in the low nibble
//                         of byte i, element 2i + 1 in the high one;
//   vscale  2 bf16        scale s and zero point z; the value is c s + z.
// Rows lie [pages][heads][page], so a head's tokens of one page are one
// contiguous run in each of the three arrays.
#pragma once
#include <cfloat>

#include "had_common.cuh"

namespace had {

struct CacheView {
    uint32_t *kbits;
    uint8_t *vcodes;
    uint32_t *vscale;      // low half s, high half z
    int pages, heads;
    int page_log;          // log2 of the tokens of a page
};

// Row of (page, head, slot) in the three arrays; 64 bits, a pool may hold
// more than 2^31 rows.
__device__ __forceinline__ long long cache_row(const CacheView &c, int page, int head, int slot)
{
    return (((long long)page * c.heads + head) << c.page_log) + slot;
}

// The largest bf16 not above the finite x, as fp32: cut towards zero, and one
// step away from zero for a negative x that the cut moved.
__device__ __forceinline__ float bf16_down(float x)
{
    const uint32_t raw = __float_as_uint(x);
    uint32_t cut = raw & 0xffff0000u;
    if ((raw >> 31) && cut != raw) cut += 0x10000u;
    return __uint_as_float(cut);
}

constexpr int kCacheLanes = 16;        // threads of one (token, head) row

template <typename T, int E>
__device__ __forceinline__ void load_slice(const T *p, float (&v)[E])
{
    if constexpr (sizeof(T) == 2 && E == 4) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
        v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    } else if constexpr (sizeof(T) == 2) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
        v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(p + i));
            v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
        }
    }
}

// Position and page of the token `t` of sequence `b`: false where the token
// is none of the sequence's `count`, or its place is not in the table.
__device__ __forceinline__ bool cache_place(const CacheView &c, const int32_t *table,
                                            int max_pages, const int32_t *start,
                                            const int32_t *counts, int b, int t, int T,
                                            int &page, int &slot, int32_t *status)
{
    int count = counts ? __ldg(counts + b) : T;
    if (count < 0 || count > T) {
        flag(status, HAD_ERR_INVALID_ARG);
        count = count < 0 ? 0 : T;
    }
    if (t >= count) return false;
    const long long pos = (long long)__ldg(start + b) + t;
    if (pos < 0 || pos >= (long long)max_pages << c.page_log) {
        flag(status, HAD_ERR_INVALID_ARG);
        return false;
    }
    page = __ldg(table + (long long)b * max_pages + (pos >> c.page_log));
    slot = (int)(pos & ((1 << c.page_log) - 1));
    if (page < 0 || page >= c.pages) {
        flag(status, HAD_ERR_INVALID_ARG);
        return false;
    }
    return true;
}

// Tokens into the cache.  Signs: x / sigma < 0 (IEEE fp32), packed.  Values,
// all steps in IEEE fp32: z = the row's minimum rounded down to bf16, s = the
// quotient (max - z) / 15 rounded up to bf16, c = (v - z) / s rounded to the
// nearest whole number (even on ties) and clamped to [0, 15]; s and z are
// rounded outwards so that no value lies beyond code 15 by more than the
// rounding of the quotient.  s = 0 (a constant row that bf16 holds) gives
// codes 0.  A row with a NaN or an infinity, or whose z, s or range is not
// finite, gets s = z = NaN and codes 0: whoever keeps it sees NaN.
//
// HBM-bound: 2 d elements read, d/8 + d/2 + 4 bytes written per row.  16
// lanes take a row, so that a bf16 row of d = 128 is one 16-byte load per
// lane; the extremes are joined by four shuffles and a word of signs by the
// 32 / E lanes that hold its elements (E = d / 16 elements per lane).
template <typename T, int D>
__global__ void __launch_bounds__(256)
cache_append_kernel(const T *__restrict__ K, const T *__restrict__ V,
                    const float *__restrict__ sigma, CacheView c,
                    const int32_t *__restrict__ table, int max_pages,
                    const int32_t *__restrict__ start, const int32_t *__restrict__ counts,
                    int tokens, unsigned rows, int32_t *status)
{
    constexpr int E = D / kCacheLanes;
    const int lane = threadIdx.x & 31;
    const int l = lane & (kCacheLanes - 1);
    const unsigned row = (blockIdx.x * 256u + threadIdx.x) / kCacheLanes;
    const unsigned half = 0xffffu << (lane & 16);     // the lanes of this row
    if (row >= rows) return;
    const unsigned bh = row / (unsigned)tokens;
    const int t = (int)(row - bh * (unsigned)tokens);
    const int b = (int)(bh / (unsigned)c.heads), h = (int)(bh - (unsigned)b * c.heads);
    const SignRule rule = sign_rule(__ldg(sigma + h));
    if (rule.bad && l == 0) flag(status, HAD_ERR_BAD_SIGMA);
    int page, slot;
    if (!cache_place(c, table, max_pages, start, counts, b, t, tokens, page, slot, status)) return;
    const long long at = cache_row(c, page, h, slot);
    const long long from = (long long)row * D + l * E;
    float k[E], v[E];
    load_slice<T, E>(K + from, k);
    load_slice<T, E>(V + from, v);

    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) word |= negative_bit(k[i], rule) << i;
    constexpr int kPerWord = 32 / E;
    word <<= E * (l & (kPerWord - 1));
#pragma unroll
    for (int o = 1; o < kPerWord; o <<= 1) word |= __shfl_xor_sync(half, word, o);
    if ((l & (kPerWord - 1)) == 0) c.kbits[at * (D / 32) + l / kPerWord] = word;

    float lo = v[0], hi = v[0];
    bool fine = true;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        fine &= fabsf(v[i]) <= FLT_MAX;
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
    }
#pragma unroll
    for (int o = 1; o < kCacheLanes; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(half, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(half, hi, o));
    }
    fine = __all_sync(half, fine);
    const float z = bf16_down(lo + 0.0f);             // -0 becomes +0
    const float s = -bf16_down(-__fdiv_rn(hi - z, 15.0f)) + 0.0f;
    fine &= fabsf(z) <= FLT_MAX && 15.0f * s <= FLT_MAX;
    uint32_t codes = 0;
    if (fine && s > 0.0f) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float q = rintf(__fdiv_rn(v[i] - z, s));
            codes |= (uint32_t)fminf(fmaxf(q, 0.0f), 15.0f) << (4 * i);
        }
    }
    if constexpr (E == 8)
        reinterpret_cast<uint32_t *>(c.vcodes)[at * kCacheLanes + l] = codes;
    else
        reinterpret_cast<uint16_t *>(c.vcodes)[at * kCacheLanes + l] = (uint16_t)codes;
    if (l == 0)
        c.vscale[at] = fine ? (__float_as_uint(s) >> 16) | (__float_as_uint(z) & 0xffff0000u)
                            : 0x7fc07fc0u;
}

// Tokens of the cache as packed signs and fp32 values c s + z (one FMA:
// rounded once); zeros for tokens beyond a sequence's count.  HBM-bound by
// the 4 d bytes written per row; 16 lanes a row, each one load of codes and
// 16-byte stores.
template <int D>
__global__ void __launch_bounds__(256)
cache_read_kernel(CacheView c, const int32_t *__restrict__ table, int max_pages,
                  const int32_t *__restrict__ start, const int32_t *__restrict__ counts,
                  int tokens, unsigned rows, uint32_t *__restrict__ bits,
                  float *__restrict__ values, int32_t *status)
{
    constexpr int E = D / kCacheLanes;
    const int l = threadIdx.x & (kCacheLanes - 1);
    const unsigned row = (blockIdx.x * 256u + threadIdx.x) / kCacheLanes;
    if (row >= rows) return;
    const unsigned bh = row / (unsigned)tokens;
    const int t = (int)(row - bh * (unsigned)tokens);
    const int b = (int)(bh / (unsigned)c.heads), h = (int)(bh - (unsigned)b * c.heads);
    int page, slot;
    const bool have = cache_place(c, table, max_pages, start, counts, b, t, tokens, page, slot, status);
    const long long at = have ? cache_row(c, page, h, slot) : 0;
    if (bits && l < D / 32) bits[(long long)row * (D / 32) + l] = have ? c.kbits[at * (D / 32) + l] : 0u;
    if (!values) return;
    uint32_t codes = 0, sz = 0;
    if (have) {
        if constexpr (E == 8)
            codes = reinterpret_cast<const uint32_t *>(c.vcodes)[at * kCacheLanes + l];
        else
            codes = reinterpret_cast<const uint16_t *>(c.vcodes)[at * kCacheLanes + l];
        sz = c.vscale[at];
    }
    const float s = bf16_lo(sz), z = bf16_hi(sz);
    float4 *out = reinterpret_cast<float4 *>(values + (long long)row * D + l * E);
#pragma unroll
    for (int i = 0; i < E; i += 4) {
        float4 f;
        f.x = fmaf((float)(codes >> (4 * i) & 15u), s, z);
        f.y = fmaf((float)(codes >> (4 * i + 4) & 15u), s, z);
        f.z = fmaf((float)(codes >> (4 * i + 8) & 15u), s, z);
        f.w = fmaf((float)(codes >> (4 * i + 12) & 15u), s, z);
        out[i / 4] = f;
    }
}

}  // namespace had
