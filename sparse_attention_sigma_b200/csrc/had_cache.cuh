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

// Row of (page, head, slot) in the three arrays: below 2^32 - 1 in every pool.
constexpr uint32_t kNoRow = 0xffffffffu;

__device__ __forceinline__ uint32_t cache_row(const CacheView &c, int page, int head, int slot)
{
    return (((unsigned)page * (unsigned)c.heads + (unsigned)head) << c.page_log) + (unsigned)slot;
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

// min and max of three that give NaN when an operand is NaN
__device__ __forceinline__ float min_nan(float a, float b, float c)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two fp32 values that take one instruction together, each rounded as alone.
struct Two {
    unsigned long long raw;
    __device__ __forceinline__ Two(float a, float b)
    {
        asm("mov.b64 %0, {%1, %2};" : "=l"(raw) : "f"(a), "f"(b));
    }
    __device__ __forceinline__ explicit Two(unsigned long long r) : raw(r) {}
    __device__ __forceinline__ void get(float &a, float &b) const
    {
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(raw));
    }
};

__device__ __forceinline__ Two operator+(Two a, Two b)
{
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.raw), "l"(b.raw));
    return Two(r);
}

__device__ __forceinline__ Two operator*(Two a, Two b)
{
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.raw), "l"(b.raw));
    return Two(r);
}

__device__ __forceinline__ Two fma(Two a, Two b, Two c)
{
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a.raw), "l"(b.raw), "l"(c.raw));
    return Two(r);
}

// Division of n < 2^31 by a divisor known on the host, with the multiplier
// m = floor(2^32 (2^s - d) / d) + 1, s = ceil(log2 d): q = (hi(n m) + n) >> s
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994).
struct Divisor {
    unsigned d, mul, shift;
};

inline Divisor divisor(unsigned d)
{
    unsigned s = 0;
    while (s < 31 && (1u << s) < d) ++s;
    return Divisor{d, (unsigned)((((1ull << s) - d) << 32) / d + 1), s};
}

__device__ __forceinline__ unsigned divide(unsigned n, const Divisor &d)
{
    return (__umulhi(n, d.mul) + n) >> d.shift;
}

constexpr int kCacheLanes = 4;         // threads of one (token, head) row
constexpr int kCacheRows = 1;          // rows of a thread whose loads are in flight together

// Where the tokens of an append or a read lie: row i of rows = (b, head, t).
struct CacheTokens {
    const int32_t *table, *start, *counts;
    int max_pages, tokens;
    unsigned rows;
    Divisor per_head, heads;
};

// Row i of them: its sequence, head and token; `real`: one of the sequence's.
struct CacheToken {
    int b, head, t;
    bool real;
};

__device__ __forceinline__ CacheToken cache_token(const CacheTokens &k, unsigned i, int32_t *status)
{
    CacheToken x{0, 0, 0, false};
    if (i >= k.rows) return x;
    const unsigned bh = divide(i, k.per_head), b = divide(bh, k.heads);
    x.b = (int)b;
    x.head = (int)(bh - b * k.heads.d);
    x.t = (int)(i - bh * k.per_head.d);
    const int count = k.counts ? __ldg(k.counts + b) : k.tokens;
    if (count < 0 || count > k.tokens) flag(status, HAD_ERR_INVALID_ARG);
    x.real = x.t < count;
    return x;
}

// Row of the pool that holds a real token, none where the table has no place for it.
__device__ __forceinline__ uint32_t cache_place(const CacheView &c, const CacheTokens &k,
                                                 const CacheToken &x, int32_t *status)
{
    if (!x.real) return kNoRow;
    const long long pos = (long long)__ldg(k.start + x.b) + x.t;
    int page = -1;
    if (pos >= 0 && pos < (long long)k.max_pages << c.page_log)
        page = __ldg(k.table + (long long)x.b * k.max_pages + (pos >> c.page_log));
    if (page < 0 || page >= c.pages) {
        flag(status, HAD_ERR_INVALID_ARG);
        return kNoRow;
    }
    return cache_row(c, page, x.head, (int)(pos & ((1 << c.page_log) - 1)));
}

// E = 8 or 16 consecutive elements of a row, by 16-byte loads.
template <typename T, int E>
struct CacheSlice {
    static constexpr int kWords = sizeof(T) * E / 4;
    uint32_t raw[kWords];

    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p) + i / 4);
            raw[i] = u.x; raw[i + 1] = u.y; raw[i + 2] = u.z; raw[i + 3] = u.w;
        }
    }

    __device__ __forceinline__ float at(int i) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(raw[i]);
        else return i & 1 ? bf16_hi(raw[i / 2]) : bf16_lo(raw[i / 2]);
    }

    // bit i: element i / sigma < 0 (IEEE fp32)
    __device__ __forceinline__ uint32_t signs(const SignRule &rule, uint32_t kge) const
    {
        uint32_t bits = 0;
        bool unsure = !rule.fast;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < kWords; i += 2) {
                uint32_t neg, uns;
                bf16_signs4(raw[i], raw[i + 1], kge, neg, uns);
                bits |= flags4(neg) << (2 * i);
                unsure |= uns != 0u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                bits |= (uint32_t)(at(i) <= -rule.thr) << i;
                unsure |= at(i) < 0.0f && at(i) > -rule.thr;
            }
        }
        if (unsure) {
            bits = 0;
#pragma unroll
            for (int i = 0; i < E; ++i) bits |= negative_bit(at(i), rule) << i;
        }
        return bits;
    }
};

// Tokens into the cache.  Signs: x / sigma < 0 (IEEE fp32), packed.  Values,
// all steps in IEEE fp32: z = the row's minimum rounded down to bf16, s = the
// quotient (max - z) / 15 rounded up to bf16, c = (v - z) / s rounded to the
// nearest whole number (even on ties); s and z are rounded outwards, so a
// quotient lies in [0, 15 (1 + 2^-23)] and needs no clamp.  s = 0 (a constant
// row that bf16 holds) gives codes 0.  A row with a NaN or an infinity, or
// whose z, 15 s or 15 s + z is not finite, gets s = z = NaN and codes 0: whoever
// keeps it sees NaN.
//
// HBM-bound once the arithmetic is lean: 2 d elements read, d/8 + d/2 + 4
// bytes written per row.  4 lanes take a row: what a row costs once (place,
// scale, checks: about 200 instructions) is shared by E = d / 4 elements a lane.
// The extremes are joined by two shuffles and a word of signs by the 32 / E lanes
// that hold its elements.  Element-wise arithmetic takes two values an
// instruction.  A quotient is x y with y = 1 / s rounded, corrected once by its
// exact remainder (P. Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990); it has the nearest whole number of the
// IEEE quotient: s has 8 bits and a half of a code 5, so x is their product
// exactly or x / s is more than half a unit in the last place away from it, and
// the corrected quotient is off by less than 2^-46.  No lane leaves early: the
// shuffles then name the whole warp, and half-warp masks cost more than all of
// the arithmetic.  229 k rows of d 128,
// bf16: 80 us with those, 57 us with whole warps and 16 lanes a row, 46 us with 8
// and a division beside each half, 36 us without, 29 us now; 21 us of HBM time.
template <typename T, int D>
__global__ void __launch_bounds__(256)
cache_append_kernel(const T *__restrict__ K, const T *__restrict__ V,
                    const float *__restrict__ sigma, CacheView c, CacheTokens k, int32_t *status)
{
    constexpr int E = D / kCacheLanes, kPerWord = 32 / E;
    const int l = threadIdx.x & (kCacheLanes - 1);
    const unsigned step = gridDim.x * (256u / kCacheLanes);
    const unsigned row0 = blockIdx.x * (256u / kCacheLanes) + threadIdx.x / kCacheLanes;    // (threads pass 2^32)
    CacheSlice<T, E> key[kCacheRows], value[kCacheRows];
    CacheToken token[kCacheRows];
    uint32_t at[kCacheRows];
    float sg[kCacheRows];
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) token[i] = cache_token(k, row0 + i * step, status);
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
        // (a token that is not there reads the first row: it is in the cache)
        const long long row = token[i].real ? row0 + i * step : 0;
        key[i].load(K + row * D + l * E);
        value[i].load(V + row * D + l * E);
        sg[i] = __ldg(sigma + token[i].head);
    }
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) at[i] = cache_place(c, k, token[i], status);
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
        const bool here = at[i] != kNoRow;
        const SignRule rule = sign_rule(sg[i]);
        if (rule.bad && l == 0 && here) flag(status, HAD_ERR_BAD_SIGMA);
        uint32_t word = key[i].signs(rule, bf16_kge(rule)) << (E * (l & (kPerWord - 1)));
#pragma unroll
        for (int o = 1; o < kPerWord; o <<= 1) word |= __shfl_xor_sync(kFullMask, word, o);
        if (here && (l & (kPerWord - 1)) == 0) c.kbits[(size_t)at[i] * (D / 32) + l / kPerWord] = word;

        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = value[i].at(e);
        float lo = v[0], hi = v[0];
#pragma unroll
        for (int e = 1; e < E; e += 2) {
            lo = min_nan(lo, v[e], v[e + 1 < E ? e + 1 : e]);
            hi = max_nan(hi, v[e], v[e + 1 < E ? e + 1 : e]);
        }
#pragma unroll
        for (int o = 1; o < kCacheLanes; o <<= 1) {
            const float l2 = __shfl_xor_sync(kFullMask, lo, o), h2 = __shfl_xor_sync(kFullMask, hi, o);
            lo = min_nan(lo, l2, l2);
            hi = max_nan(hi, h2, h2);
        }
        const float z = bf16_down(lo + 0.0f);         // -0 becomes +0
        const float s = -bf16_down(-__fdiv_rn(hi - z, 15.0f)) + 0.0f;
        const bool fine = fabsf(lo) <= FLT_MAX && fabsf(hi) <= FLT_MAX && fabsf(z) <= FLT_MAX &&
                          15.0f * s <= FLT_MAX && fmaf(15.0f, s, z) <= FLT_MAX;
        const bool coded = fine && s > 0.0f;
        const float inv = __frcp_rn(s);
        // four codes c0 + 16 c1 + 256 c2 + 4096 c3 are a whole number below
        // 2^16, exact in fp32, and the last bits of its sum with 2^23
        constexpr float kWhole = 12582912.0f;         // 1.5 2^23: the sum's last bit is 1
        const Two minus_z(-z, -z), by(inv, inv), up(kWhole, kWhole), down(-kWhole, -kWhole);
        const Two minus_s(-s, -s);
        uint32_t codes[E / 8];
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            float r[4];
#pragma unroll
            for (int f = 0; f < 4; f += 2) {
                const Two x = Two(v[e + f], v[e + f + 1]) + minus_z, q = x * by;
                (fma(fma(q, minus_s, x), by, q) + up + down).get(r[f], r[f + 1]);
            }
            const float four = fmaf(fmaf(r[3], 16.0f, r[2]), 256.0f, fmaf(r[1], 16.0f, r[0]));
            const uint32_t low = __float_as_uint(four + 8388608.0f);
            codes[e / 8] = e % 8 ? __byte_perm(codes[e / 8], low, 0x5410) : low;
        }
        if (coded && s < 8.077936e-28f) {             // 2^-90: a remainder may be subnormal
#pragma unroll
            for (int e = 0; e < E; ++e)
                codes[e / 8] = (e % 8 ? codes[e / 8] : 0u) |
                               (uint32_t)rintf(__fdiv_rn(v[e] - z, s)) << (4 * (e % 8));
        }
        if (here) {
            uint32_t *const to = reinterpret_cast<uint32_t *>(c.vcodes) + (size_t)at[i] * (D / 8) + l * (E / 8);
            if constexpr (E == 32)
                *reinterpret_cast<uint4 *>(to) = coded ? make_uint4(codes[0], codes[1], codes[2], codes[3])
                                                       : make_uint4(0u, 0u, 0u, 0u);
            else
                *reinterpret_cast<uint2 *>(to) = coded ? make_uint2(codes[0], codes[1]) : make_uint2(0u, 0u);
            if (l == 0)
                c.vscale[at[i]] = fine ? (__float_as_uint(s) >> 16) | (__float_as_uint(z) & 0xffff0000u)
                                       : 0x7fc07fc0u;
        }
    }
}

// Tokens of the cache as packed signs and fp32 values c s + z (one FMA:
// rounded once); zeros for tokens beyond a sequence's count.  HBM-bound by
// the 4 d bytes written per row; 8 lanes a row, each D / 32 times 16 bytes of
// consecutive lanes, two rows in flight (262 k rows of d 128, of which 229 k are
// there: 27 us, with 16 lanes a row 30 us; 24 us of HBM time).
constexpr int kReadLanes = 8, kReadRows = 2;

template <int D>
__global__ void __launch_bounds__(256)
cache_read_kernel(CacheView c, CacheTokens k, uint32_t *__restrict__ bits,
                  float *__restrict__ values, int32_t *status)
{
    constexpr int E = D / kReadLanes;
    const int l = threadIdx.x & (kReadLanes - 1);
    const unsigned step = gridDim.x * (256u / kReadLanes);
    const unsigned row0 = blockIdx.x * (256u / kReadLanes) + threadIdx.x / kReadLanes;    // (threads pass 2^32)
    uint32_t at[kReadRows];
    uint32_t codes[kReadRows][E / 4], sz[kReadRows], word[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i)
        at[i] = cache_place(c, k, cache_token(k, row0 + i * step, status), status);
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        const bool here = at[i] != kNoRow;
        word[i] = here && bits && l < D / 32 ? __ldg(c.kbits + (size_t)at[i] * (D / 32) + l) : 0u;
        sz[i] = here && values ? __ldg(c.vscale + at[i]) : 0u;
#pragma unroll
        for (int e = 0; e < E / 4; ++e)
            codes[i][e] = here && values ? __ldg(reinterpret_cast<const uint16_t *>(c.vcodes) +
                                                 (size_t)at[i] * (D / 4) + e * kReadLanes + l) : 0u;
    }
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        const unsigned row = row0 + i * step;
        if (row >= k.rows) break;
        if (bits && l < D / 32) bits[(long long)row * (D / 32) + l] = word[i];
        if (!values) continue;
        const Two s(bf16_lo(sz[i]), bf16_lo(sz[i])), z(bf16_hi(sz[i]), bf16_hi(sz[i]));
        // 2^23 + c has c in its last bits
        const Two down(-8388608.0f, -8388608.0f);
        auto raised = [](uint32_t code) { return __uint_as_float((code & 15u) | 0x4b000000u); };
#pragma unroll
        for (int e = 0; e < E / 4; ++e) {
            const uint32_t x = codes[i][e];
            float4 f;
            fma(Two(raised(x), raised(x >> 4)) + down, s, z).get(f.x, f.y);
            fma(Two(raised(x >> 8), raised(x >> 12)) + down, s, z).get(f.z, f.w);
            reinterpret_cast<float4 *>(values + (long long)row * D)[e * kReadLanes + l] = f;
        }
    }
}

}  // namespace had
