// had_cache_attn.cuh -- attention of new tokens to the decoder cache.
//
// Row (b, h, t) sits at position i = len_b - count_b + t of its sequence and
// sees the cached tokens j <= i, under a window W > 0 only those with
// j > i - W or j < S (the first S tokens stay visible).  Of the visible ones
// it keeps the n = min(N, visible) with the smallest Hamming distance h_j (the
// largest logit s_j = d - 2 h_j), the lower j on ties, and
//   out = sum_kept p_j (c_j s_j + z_j),  p = softmax(tau (d - 2 h)) over them.
// A logit is one of d + 1 levels, so the row's histogram of distances gives
// the threshold level, the ties kept on it, the largest logit and the sum Z
// of the softmax before any value is read: p_j is a table lookup by h_j, and
// partial sums over parts of the keys just add up.
//
// One cluster of CTAs takes a tile of R rows that share a key-value head (its
// query heads, and neighbouring tokens of a draft or chunk) and splits the keys
// that any of them sees; a CTA's four warps split its slice, in key order.
//   1. Distances: a lane per key, the key's bits in registers, XOR + popc with
//      every row's bits from shared memory; 8-bit distances stay in shared
//      memory (d + 1: not visible), counts go to the CTA's histograms.
//   2. The cluster's histograms are read through distributed shared memory; a
//      warp per row finds level, quota and Z and fills p[h].  The ties that
//      lower-ranked CTAs hold come from the same counts.
//   3. Each warp goes through its part again, drops what a row does not keep
//      (ties by rank in key order) and queues the keys that at least one row
//      keeps; their codes and scales are copied to shared memory from there.
//   4. Per 16 queued keys, behind their copies: the tile's P V on the tensor
//      core.  The codes are whole numbers below 16, exact in fp16; the weights
//      p s are fp32, brought into fp16's range by a power of two per row that
//      only comes down when a larger weight appears, and cut into two fp16
//      terms, stacked as rows of A: row x = 8 term + r.  The terms are off by
//      2^-23 of their weight at most, or by 2^-37 of the row's largest weight
//      p s, for scales of any size.  The product takes c - 8 in place of c; the
//      rest, p (z + 8 s), is summed beside it, so an element's error is measured
//      by sum p (8 s + |z + 8 s|): far below the values' own step s.
//   5. Warps, terms and CTAs are added in a fixed order.
// The union of the rows' kept keys is read once, each key's bits once.
//
// mma.sync and not tcgen05: a tile has 4 or 8 rows of 64 or 128, B is made in
// registers from gathered codes, and the tensor pipe is 10 % busy.  What bounds
// it is the instructions around the product and their latency at 16 warps an SM
// (16 sequences of 16 k tokens, 32 query and 8 key heads, d 128, N 2048: 67 us,
// 31 M warp instructions in half of the issue slots; 127 MB from memory would
// take 19 us): about 20 a (row, 32 keys) for distances and selection, 300 per 16 kept keys
// of d 128, of which 100 unpack and multiply codes, 70 make the weights and 40
// copy.  The accumulators' registers allow 16 warps an SM at d 128 and 20 to 24
// at 64; more spill (20 and 24 at d 128, with the bf16 form of step 4: 95 and
// 115 us against 72), fewer hide less (12: 92 us).  Loops over rows and over
// the first copies are kept rolled: unrolled, the kernel passes what the SM
// holds of instructions (windowed chunks 141 against 125 us).
#pragma once
#include <cooperative_groups.h>

#include "had_cache.cuh"

namespace had {

namespace cg = cooperative_groups;

struct CacheAttnArgs {
    const void *Q;
    bool q_bf16;                       // else fp32
    const float *sigma;
    CacheView c;
    const int32_t *table, *lens, *counts;
    int max_pages, Hq, T, N, window, sinks;
    float tau;
    float *out;
    int32_t *status;
};

// Visible keys of a row: [0, sinks) and [lo, pos]; pos = -1 for none.
struct RowRange {
    int sinks, lo, pos;
};

__device__ __forceinline__ RowRange row_range(const CacheAttnArgs &a, int len, int count, int t)
{
    RowRange r;
    r.pos = t < count ? max(len - count + t, -1) : -1;
    r.lo = a.window > 0 ? max(0, r.pos - a.window + 1) : 0;
    r.sinks = min(a.sinks, r.lo);
    return r;
}

constexpr int kMaxCtas = 8;            // of a cluster
constexpr int kCacheAttnThreads = 128, kCacheAttnWarps = kCacheAttnThreads / 32;

// The tile's split: R rows, `tiles` tiles per (sequence, head), `ctas` per
// cluster at most, of which a tile uses as many as its keys ask for, `cap` keys a
// CTA holds at once (a multiple of its threads).
struct CacheAttnPlan {
    int R, tiles, ctas, cap;
    Divisor by_tiles, by_heads, by_group;      // of tiles, heads, query heads per head
};

// Entries of the list of pages under `cap` keys: two runs of keys (the first
// tokens and the window) that need not begin with a page.
__host__ __device__ constexpr int cache_attn_pages(int cap) { return cap / 16 + 4; }

// A warp's own shared memory in steps 3 and 4: the queue of kept keys (row of
// the pool, a distance per row of the tile), a ring of kStages chunks of 16
// keys (codes, rows padded by 16 bytes so that the eight lanes of a key and the
// four keys of a load fall on different banks; scales), and the stacked rows
// of A.
constexpr int kStages = 4;
constexpr int kQueue = 128;            // >= 16 (kStages + 1) + 31

template <int D, int RW>
struct WarpStage {
    static constexpr int kStride = D / 2 + 16;
    union {
        __align__(16) unsigned char codes[kStages][16 * kStride];
        int hist[4 * RW][D + 2];       // before: this warp's counts; D + 1: not seen
    };
    __align__(8) uint32_t scale[kStages][16];
    // (these three also hold a row's counts on their way from the cluster)
    uint4 terms[2][8][4];              // registers of A by lane: [g][t4]
    uint32_t pool_row[kQueue];
    __align__(8) uint32_t dist[RW][kQueue];
};

// The warps' results before they are added: [warps][16][kSumStride] floats.
// Column n of accumulator tile i is element n D/8 + i; its 16-byte piece i / 4
// lies at place (i / 4) ^ sum_swizzle(n), and a row is padded, so that the
// eight lanes of a store's wavefront (two rows, four columns) fall on different
// banks.
template <int D>
constexpr int kSumStride = D + D / 8;

template <int D>
__device__ __forceinline__ int sum_swizzle(int n)
{
    return D == 128 ? n >> 1 : n >> 2;
}

template <int D, int RW>
size_t cache_attn_smem_bytes(int cap)
{
    const size_t keys = sizeof(WarpStage<D, RW>) * kCacheAttnWarps + (size_t)cap * 4 * RW + cache_attn_pages(cap) * 4;
    const size_t sums = sizeof(float) * kCacheAttnWarps * 16 * kSumStride<D>;
    return keys > sums ? keys : sums;
}

__device__ __forceinline__ void copy_async16(void *to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :: "r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}

__device__ __forceinline__ void copy_async4(void *to, const void *from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                 :: "r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}

// A word of another CTA's shared memory, by its address in one's own.
__device__ __forceinline__ int load_of_cta(uint32_t at, int cta)
{
    uint32_t there;
    int x;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(cta));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(there) : "memory");
    return x;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Codes of two keys as fp16 c - 8, from the low (even elements) or the high
// nibbles of the low bytes of x's halves: 1024 + c and 1024 + 16 c have c in
// their mantissas, the rest is exact.  The tensor core cuts its running sums, it
// does not round them; sums of the centred codes stay near zero, those of c
// itself would grow with every key and lose bits on the way (16 k keys, N 2048:
// relative error 3.3e-6 instead of 2.2e-7).  `raised`: 0x64006400, in a register
// that the compiler does not fill anew for each use.
__device__ __forceinline__ uint32_t codes_low(uint32_t x, uint32_t raised)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"((x & 0x000f000fu) | raised), "r"(0x64086408u));
    return r;
}

__device__ __forceinline__ uint32_t codes_high(uint32_t x, uint32_t raised)
{
    uint32_t r;                        // (1024 + 16 c) / 16 - 72
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r)
        : "r"((x & 0x00f000f0u) | raised), "r"(0x2c002c00u), "r"(0xd480d480u));
    return r;
}

// Two fp32 as fp16, a in the low half; and back.
__device__ __forceinline__ uint32_t to_f16(float a, float b)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ float2 from_f16(uint32_t x)
{
    float2 r;
    asm("{.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}"
        : "=f"(r.x), "=f"(r.y) : "r"(x));
    return r;
}

// 255 in the bytes where a < b (unsigned), 0 in the others
__device__ __forceinline__ uint32_t bytes_below(uint32_t a, uint32_t b)
{
    const uint32_t t = (a | 0x80808080u) - (b & 0x7f7f7f7fu);      // bit 7 clear: low 7 bits of a less
    const uint32_t less = (~a & b) | (~(a ^ b) & ~t);              // in bit 7
    uint32_t spread;                                               // bit 7 over the byte
    asm("prmt.b32 %0, %1, %2, 0xba98;" : "=r"(spread) : "r"(less), "r"(0u));
    return spread;
}

// The largest scaled weight, and the largest scale: p 2^127 is finite.
constexpr float kMostWeight = 32768.0f;
constexpr float kMostScale = 1.7014118e38f;

template <int D, int RW>
struct CacheAttnShared {
    static constexpr int RM = 4 * RW;
    __align__(16) uint32_t qbits[RM][D / 32];
    int pos[RM], lo[RM];
    int hist[RM][D + 2];               // the counts of all warps
    union {
        float p[RM][D + 2];            // weight of a distance; 0 for D + 1
        float part[RM][D];             // at the end: this CTA's sums
    };
    int level[RM], quota[RM];
    int ranked;                        // some row keeps only part of its ties
    int ties[kCacheAttnWarps][RM];
    float zsum[kCacheAttnWarps][RM];
};

// RW: words of four distances per key, for tiles of up to 4 RW rows; RW <= 2.
// kLong: a CTA's slice may pass `cap` keys, and is then gone through twice, in
// segments.  A template parameter, since that path costs the other one registers
// (5 % of the time of 16 k keys a sequence).
template <int D, int RW, bool kLong>
__global__ void __launch_bounds__(kCacheAttnThreads, D == 128 ? 4 : RW == 2 || kLong ? 5 : 6)
cache_attn_kernel(CacheAttnArgs a, CacheAttnPlan plan)
{
    constexpr int kThreads = kCacheAttnThreads, W = kCacheAttnWarps, DW = D / 32;
    constexpr int kTiles = D / 8;             // 8-wide column tiles of the value
    constexpr int kCodeWords = D / 64;        // 32-bit words of codes per lane and key
    constexpr int RM = 4 * RW;
    constexpr uint32_t kUnseen = D + 1, kUnseen4 = kUnseen * 0x01010101u;
    constexpr int KU = 4;                     // keys per lane of one step of the distances
    using Shared = CacheAttnShared<D, RW>;
    extern __shared__ __align__(16) unsigned char attn_smem[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int R = plan.R, cap = plan.cap;
    using Stage = WarpStage<D, RW>;
    Stage &stage = reinterpret_cast<Stage *>(attn_smem)[warp];
    uint32_t *const distw = reinterpret_cast<uint32_t *>(                    // [RW][cap]
        attn_smem + sizeof(Stage) * W);
    uint32_t *const page_row = distw + RW * cap;                             // first row of a page

    const int rank = (int)(blockIdx.x & (unsigned)(plan.ctas - 1));        // a power of two
    const unsigned unit = blockIdx.x >> (__ffs(plan.ctas) - 1);
    const unsigned bh = divide(unit, plan.by_tiles), b = divide(bh, plan.by_heads);
    const int tile = (int)(unit - bh * (unsigned)plan.tiles);
    const int h = (int)(bh - b * (unsigned)a.c.heads), G = (int)plan.by_group.d;
    const int row0 = tile * R, rows = min(R, G * a.T - row0);
    const int lg = a.c.page_log, page_mask = (1 << lg) - 1;
    const int32_t *const table = a.table + (long long)b * a.max_pages;

    // row r of the tile: token (row0 + r) / G, query head h G + (row0 + r) % G
    auto token_of = [&](int r) { return (int)divide((unsigned)(row0 + r), plan.by_group); };
    auto q_row = [&](int r) -> long long {
        const int t = token_of(r), g = row0 + r - t * G;
        return ((long long)b * a.Hq + h * G + g) * a.T + t;
    };
    int len = __ldg(a.lens + b), count = a.counts ? __ldg(a.counts + b) : a.T;
    constexpr int kMine = (RM + W - 1) / W;
    float x[kMine][DW], sigma[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int r = min(warp + i * W, rows - 1);
        const long long at = q_row(r) * D + lane;
        sigma[i] = __ldg(a.sigma + h * G + row0 + r - token_of(r) * G);
#pragma unroll
        for (int w = 0; w < DW; ++w)
            x[i][w] = a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.Q)[at + 32 * w])
                               : static_cast<const float *>(a.Q)[at + 32 * w];
    }
    if (len < 0 || len > (long long)a.max_pages << lg || count < 0 || count > a.T) {
        if (tid == 0) flag(a.status, HAD_ERR_INVALID_ARG);
        len = count = 0;
    }
    // keys that some row of the tile sees: [0, first_n) and [lo, hi]
    const int t_first = token_of(0), t_last = token_of(rows - 1);
    const int t_lo = max(t_first, count - len), t_hi = min(t_last, count - 1);
    int lo = 0, first_n = 0, total = 0;
    int min_pos = -1, max_lo = 0;             // a key in [max_lo, min_pos] is seen by every row
    if (t_lo <= t_hi) {
        const RowRange from = row_range(a, len, count, t_lo), to = row_range(a, len, count, t_hi);
        lo = from.lo;
        first_n = from.sinks;
        total = first_n + to.pos + 1 - lo;
        max_lo = to.lo;
        if (t_first == t_lo && t_last == t_hi) min_pos = from.pos;
    }
    // The CTAs that this tile uses, one per 512 keys or per `cap`, which may be
    // less; the others leave at once (a cluster's barriers wait for those that are
    // there).  The host knows no lengths and launches for as many keys as a row of
    // the table may hold (one sequence of 200 tokens in a table for 128 k: 8.4 us,
    // with all eight CTAs 9.7 us).
    int C = 1;
    while (C < plan.ctas && total > min(512, cap) * C) C *= 2;
    if (rank >= C) return;

#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int r = warp + i * W;
        if (r >= rows) break;
        const SignRule rule = sign_rule(sigma[i]);
        if (rule.bad && lane == 0) flag(a.status, HAD_ERR_BAD_SIGMA);
#pragma unroll
        for (int w = 0; w < DW; ++w) {
            const uint32_t word = __ballot_sync(kFullMask, negative_bit(x[i][w], rule));
            if (lane == 0) sh.qbits[r][w] = word;
        }
    }
    if (tid == 0) sh.ranked = 0;
    for (int i = lane; i < RM * (D + 2); i += 32) (&stage.hist[0][0])[i] = 0;
    if (tid < rows) {
        const RowRange rr = row_range(a, len, count, token_of(tid));
        sh.pos[tid] = rr.pos;
        sh.lo[tid] = rr.lo;
    }

    const int first_pages = (first_n + page_mask) >> lg;
    // this CTA's slice of them, whole groups of 32
    const int per = ((total + C - 1) / C + 31) & ~31;
    const int u0 = min(total, rank * per), u1 = min(total, u0 + per);
    const int segs = kLong ? max(1, (u1 - u0 + cap - 1) / cap) : 1;

    // key u of them: its position; its page's index among the pages of all of them
    const int to_key = lo - first_n, to_page = first_pages - (lo >> lg);
    auto key_of = [&](int u) { return u < first_n ? u : u + to_key; };
    auto page_at = [&](int u) { return (key_of(u) >> lg) + (u < first_n ? 0 : to_page); };

    // Keys s0 .. s0 + n - 1 of the slice: their pages, then this warp's distances.
    auto load_pages = [&](int s0, int n) {
        if (n <= 0) return;
        const int first = page_at(s0), last = page_at(s0 + n - 1);
        for (int i = first + tid; i <= last; i += kThreads) {
            const int page = __ldg(table + (i < first_pages ? i : i - to_page));
            const bool there = page >= 0 && page < a.c.pages;
            if (!there) flag(a.status, HAD_ERR_INVALID_ARG);
            page_row[i - first] = there ? (page * (unsigned)a.c.heads + h) << lg : kNoRow;
        }
    };
    auto distances = [&](int s0, int wb, int we, bool with_hist) {
        if (wb >= we) return;
        const int page0 = page_at(s0);
        uint32_t next[KU][DW], next_row[KU];
        auto fetch = [&](int k0) {
#pragma unroll
            for (int i = 0; i < KU; ++i) {
                const int u = min(s0 + k0 + 32 * i + lane, s0 + we - 1);
                const uint32_t first = page_row[page_at(u) - page0];
                const bool have = k0 + 32 * i + lane < we && first != kNoRow;
                next_row[i] = have ? first + (key_of(u) & page_mask) : kNoRow;
#pragma unroll
                for (int w = 0; w < DW; ++w) next[i][w] = 0u;
                if (have) {
                    if constexpr (DW == 2) {
                        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(a.c.kbits) + next_row[i]);
                        next[i][0] = x.x; next[i][1] = x.y;
                    } else {
                        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(a.c.kbits) + next_row[i]);
                        next[i][0] = x.x; next[i][1] = x.y; next[i][2] = x.z; next[i][3] = x.w;
                    }
                }
            }
        };
        // 32 KU keys against all rows; `mixed`: some row may not see some key
        auto step = [&](int k0, const uint32_t (&bits)[KU][DW], const uint32_t (&at)[KU], bool mixed) {
#pragma unroll 1
            for (int q = 0; q < RW; ++q) {
                uint32_t word[KU];
#pragma unroll
                for (int i = 0; i < KU; ++i) word[i] = kUnseen4;
#pragma unroll 1
                for (int r = 4 * q; r < min(rows, 4 * q + 4); ++r) {
                    uint32_t qb[DW];
                    if constexpr (DW == 2) {
                        const uint2 x = *reinterpret_cast<const uint2 *>(sh.qbits[r]);
                        qb[0] = x.x; qb[1] = x.y;
                    } else {
                        const uint4 x = *reinterpret_cast<const uint4 *>(sh.qbits[r]);
                        qb[0] = x.x; qb[1] = x.y; qb[2] = x.z; qb[3] = x.w;
                    }
                    const int pos = mixed ? sh.pos[r] : 0, row_lo = mixed ? sh.lo[r] : 0;
                    const unsigned unit = 1u << (8 * (r & 3));
#pragma unroll
                    for (int i = 0; i < KU; ++i) {
                        if (k0 + 32 * i >= we) break;
                        int n = 0;
#pragma unroll
                        for (int w = 0; w < DW; ++w) n += __popc(bits[i][w] ^ qb[w]);
                        bool vis = at[i] != kNoRow;
                        if (mixed) {
                            const int key = key_of(s0 + k0 + 32 * i + lane);
                            vis = vis && key <= pos && (key >= row_lo || key < a.sinks);
                        }
                        n = vis ? n : (int)kUnseen;
                        word[i] += ((unsigned)n - kUnseen) * unit;
                        if (with_hist) atomicAdd(&stage.hist[r][n], 1);
                    }
                }
#pragma unroll
                for (int i = 0; i < KU; ++i) {
                    const int k = k0 + 32 * i + lane;
                    if (k < we) distw[q * cap + k] = word[i];
                }
            }
        };
        fetch(wb);
        for (int k0 = wb; k0 < we; k0 += 32 * KU) {
            uint32_t bits[KU][DW], at[KU];
#pragma unroll
            for (int i = 0; i < KU; ++i) {
                at[i] = next_row[i];
#pragma unroll
                for (int w = 0; w < DW; ++w) bits[i][w] = next[i][w];
            }
            if (k0 + 32 * KU < we) fetch(k0 + 32 * KU);
            const int k_last = min(we, k0 + 32 * KU) - 1;
            if (key_of(s0 + k_last) <= min_pos && key_of(s0 + k0) >= max_lo)
                step(k0, bits, at, false);
            else
                step(k0, bits, at, true);
        }
    };
    // a warp's part of n keys: whole groups of 32, in key order
    auto warp_begin = [&](int n, int w) { return min(n, (((n + 31) >> 5) * w / W) << 5); };

    for (int seg = 0; seg < segs; ++seg) {
        const int s0 = u0 + seg * cap, n = min(cap, u1 - s0);
        __syncthreads();                      // rows are set up; the last segment's pages are done
        load_pages(s0, n);
        __syncthreads();
        distances(s0, warp_begin(n, warp), warp_begin(n, warp + 1), true);
    }
    __syncthreads();
    for (int i = tid; i < rows * (D + 2); i += kThreads) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) n += (&reinterpret_cast<Stage *>(attn_smem)[w].hist[0][0])[i];
        (&sh.hist[0][0])[i] = n;
    }
    cg::cluster_group cluster = cg::this_cluster();
    if (C > 1) cluster.sync();
    else __syncthreads();

    // level, quota and weights: a warp per row, EL consecutive levels per lane
    for (int r = warp; r < rows; r += W) {
        constexpr int EL = (D + 2 + 31) / 32;
        int cnt[EL], before[EL], sum = 0;
#pragma unroll
        for (int e = 0; e < EL; ++e) cnt[e] = before[e] = 0;
        if (C > 1) {
            // the cluster's counts, neighbouring words by neighbouring lanes and
            // four CTAs' in flight at once, through this warp's shared memory
            // to the order in which they are added up
            int all[EL], below[EL];
#pragma unroll
            for (int e = 0; e < EL; ++e) all[e] = below[e] = 0;
            const uint32_t here = (uint32_t)__cvta_generic_to_shared(&sh.hist[r][lane]);
            for (int o0 = 0; o0 < C; o0 += 4) {
                int x[4][EL];
#pragma unroll
                for (int o = 0; o < 4; ++o)
#pragma unroll
                    for (int e = 0; e < EL; ++e)
                        x[o][e] = o0 + o < C && lane + 32 * e <= D ? load_of_cta(here + 128 * e, o0 + o) : 0;
#pragma unroll
                for (int o = 0; o < 4; ++o)
#pragma unroll
                    for (int e = 0; e < EL; ++e) {
                        all[e] += x[o][e];
                        below[e] += o0 + o < rank ? x[o][e] : 0;
                    }
            }
            int *const to = reinterpret_cast<int *>(&stage.terms);          // 64 EL words
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                to[lane + 32 * e] = all[e];
                to[32 * EL + lane + 32 * e] = below[e];
            }
            __syncwarp();
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                cnt[e] = to[lane * EL + e];
                before[e] = to[32 * EL + lane * EL + e];
            }
            __syncwarp();
        } else {
#pragma unroll
            for (int e = 0; e < EL; ++e) cnt[e] = lane * EL + e <= D ? sh.hist[r][lane * EL + e] : 0;
        }
#pragma unroll
        for (int e = 0; e < EL; ++e) sum += cnt[e];
        int upto = sum;                       // inclusive prefix over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFullMask, upto, o);
            if (lane >= o) upto += x;
        }
        const int seen = __shfl_sync(kFullMask, upto, 31), n = min(a.N, seen);
        int cum = upto - sum, level = -1, quota = 0, first = D + 1;
#pragma unroll
        for (int e = 0; e < EL; ++e) {
            if (cnt[e] > 0 && first > D) first = lane * EL + e;
            if (cum < n && n <= cum + cnt[e]) {
                level = lane * EL + e;
                quota = n - cum;
                sh.quota[r] = max(0, quota - before[e]);
                if (quota < cnt[e]) sh.ranked = 1;
            }
            cum += cnt[e];
        }
        first = __reduce_min_sync(kFullMask, first);
        const int owner = __reduce_max_sync(kFullMask, level >= 0 ? lane : -1);
        level = __shfl_sync(kFullMask, level, max(owner, 0));
        quota = __shfl_sync(kFullMask, quota, max(owner, 0));
        // exp(tau (s_l - s_first)) = 2^(2 tau log2(e) (first - l)); a tau so large
        // that the product overflows leaves the first level alone, as it should
        const float rate = fminf(2.8853901f * a.tau, FLT_MAX);
        float w[EL], z = 0.0f;
#pragma unroll
        for (int e = 0; e < EL; ++e) {
            const int l = lane * EL + e;
            w[e] = l <= level && cnt[e] > 0 ? exp2f(rate * (float)(first - l)) : 0.0f;
            z += w[e] * (float)(l < level ? cnt[e] : quota);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFullMask, z, o);
        const float inv = z > 0.0f ? __frcp_rn(z) : 0.0f;
#pragma unroll
        for (int e = 0; e < EL; ++e)
            if (lane * EL + e <= D + 1) sh.p[r][lane * EL + e] = lane * EL + e <= D ? w[e] * inv : 0.0f;
        if (lane == 0) {
            sh.level[r] = level;
            if (level < 0) sh.quota[r] = 0;
        }
    }
    __syncthreads();

    const int g = lane >> 2, t4 = lane & 3;
    uint32_t raised;
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(raised));
    // scale[i]: the power of two by which row 4 i + lane / 8 is multiplied
    float acc[kTiles][4], zacc[RW], scale[RW], shrink[RW];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        zacc[i] = 0.0f;
        scale[i] = kMostScale;
        shrink[i] = 1.0f;
    }
    // rows that the tile lacks stay zero
    for (int i = lane; i < 2 * 32; i += 32) (&stage.terms[0][0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
    // the factor of row g among those of the rows 4 i + lane / 8
    auto of_row_g = [&](const float (&x)[RW]) {
        float f = __shfl_sync(kFullMask, x[0], (g & 3) * 8);
        if constexpr (RW == 2) {
            const float f1 = __shfl_sync(kFullMask, x[1], (g & 3) * 8);
            f = g < 4 ? f : f1;
        }
        return f;
    };
    // what was summed under the rows' scales of before
    auto shrink_sums = [&]() {
        const float f = of_row_g(shrink);
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] *= f;
    };
    // lane r < rows follows row r's level and the ties it may still keep
    const int my_level = lane < rows ? sh.level[lane] : -1;
    int my_quota = lane < rows ? sh.quota[lane] : 0;

    for (int seg = 0; seg < segs; ++seg) {
        const int s0 = u0 + seg * cap, n = min(cap, u1 - s0);
        const int wb = warp_begin(n, warp), we = warp_begin(n, warp + 1);
        if (kLong && segs > 1) {              // the slice did not fit: again from the bits
            __syncthreads();
            load_pages(s0, n);
            __syncthreads();
            distances(s0, wb, we, false);
        }
        // ties of each row in this warp's part, where a row keeps only some
        int before = 0, all = 0, here = 0;
        if (!kLong && sh.ranked && lane < rows && my_level >= 0) {
            for (int w = 0; w < W; ++w) {
                const int x = reinterpret_cast<Stage *>(attn_smem)[w].hist[lane][my_level];
                before += w < warp ? x : 0;
                here = w == warp ? x : here;
            }
        }
        if (!kLong) __syncthreads();          // the counts make room for the copies
        if (kLong && sh.ranked) {             // counts of one segment
            for (int q = 0; q < RW; ++q) {
                uint32_t same = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int l = __shfl_sync(kFullMask, my_level, 4 * q + i);
                    same |= (l < 0 ? 0xffu : (uint32_t)l) << (8 * i);
                }
                uint32_t mine = 0;                // a byte per row: at most cap / 128 + 1 keys a lane
                for (int k = wb + lane; k < we; k += 32)
                    mine += __vcmpeq4(distw[q * cap + k], same) & 0x01010101u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int s = __reduce_add_sync(kFullMask, mine >> (8 * i) & 255u);
                    if (lane == 0 && 4 * q + i < rows) sh.ties[warp][4 * q + i] = s;
                }
            }
            __syncthreads();
            if (lane < rows) {
                for (int w = 0; w < W; ++w) {
                    const int x = sh.ties[w][lane];
                    before += w < warp ? x : 0;
                    all += x;
                    here = w == warp ? x : here;
                }
            }
        }
        // keep bytes below `limit`; a row whose quota ends inside this part
        // keeps its first `left` ties
        int left = my_quota - before;
        const bool partial = left > 0 && left < here;
        const int limit = my_level < 0 ? 0 : my_level + (left >= here);   // (unranked: all ties)
        my_quota = max(0, my_quota - all);
        const unsigned partial_rows = __ballot_sync(kFullMask, partial);
        uint32_t below[RW];
#pragma unroll
        for (int q = 0; q < RW; ++q) {
            below[q] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                below[q] |= (uint32_t)__shfl_sync(kFullMask, limit, 4 * q + i) << (8 * i);
        }
        const int page0 = n > 0 ? page_at(s0) : 0;
        int queued = 0, k0 = wb;
        // the next 32 keys of the part
        auto look = [&]() {
            const int k = k0 + lane;
            uint32_t any = 0, d4[RW];
#pragma unroll
            for (int q = 0; q < RW; ++q) {
                d4[q] = k < we ? distw[q * cap + k] : kUnseen4;
                uint32_t keep = bytes_below(d4[q], below[q]);
                for (unsigned todo = partial_rows >> (4 * q) & 15u; todo; todo &= todo - 1) {
                    const int i = __ffs(todo) - 1, r = 4 * q + i;
                    const int l = __shfl_sync(kFullMask, my_level, r);
                    const int room = __shfl_sync(kFullMask, left, r);
                    const bool tie = (int)(d4[q] >> (8 * i) & 255u) == l;
                    const unsigned ties = __ballot_sync(kFullMask, tie);
                    if (tie && __popc(ties & ((1u << lane) - 1)) < room) keep |= 255u << (8 * i);
                    if (lane == r) left -= min(left, __popc(ties));
                }
                d4[q] = (d4[q] & keep) | (kUnseen4 & ~keep);
                any |= keep;
            }
            const unsigned kept = __ballot_sync(kFullMask, any != 0u);
            if (any) {
                const int to = (queued + __popc(kept & ((1u << lane) - 1))) % kQueue, u = s0 + k;
                stage.pool_row[to] = page_row[page_at(u) - page0] + (key_of(u) & page_mask);
#pragma unroll
                for (int q = 0; q < RW; ++q) stage.dist[q][to] = d4[q];
            }
            queued += __popc(kept);
            k0 += 32;
            if (k0 >= we && queued > 0) {
                // the last chunk repeats its last key, which then weighs nothing
                __syncwarp();
                const int to = queued + lane;
                if (lane < (-queued & 15)) {
                    stage.pool_row[to % kQueue] = stage.pool_row[(queued - 1) % kQueue];
#pragma unroll
                    for (int q = 0; q < RW; ++q) stage.dist[q][to % kQueue] = kUnseen4;
                }
            }
        };
        // copies of the c-th 16 queued keys: 16-byte pieces of their codes, and scales
        constexpr int kPieces = D / 32;
        auto issue = [&](int c) {
            if (16 * c < queued) {
                const int ring = c % kStages;
                const uint32_t *const from = stage.pool_row + 16 * c % kQueue;
                unsigned char *const to = stage.codes[ring] + lane / kPieces * Stage::kStride + lane % kPieces * 16;
#pragma unroll
                for (int i = 0; i < 16 * kPieces / 32; ++i)
                    copy_async16(to + i * (32 / kPieces) * Stage::kStride,
                                 a.c.vcodes + (size_t)from[i * (32 / kPieces) + lane / kPieces] * (D / 2) +
                                     lane % kPieces * 16);
                if (lane < 16) copy_async4(&stage.scale[ring][lane], a.c.vscale + from[lane]);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // The same where a scale is NaN or a weight passes fp16's range: the rows'
        // scales come down so that the largest weight of the chunk is below 2^13
        // (four times more may come before the next time),
        // and p z is summed again with what is kept alone.
        auto reweigh = [&](int c, float (&v_a)[RW], float (&v_b)[RW], const float (&zkeep)[RW]) -> bool {
            const int pair = lane & 7, sub = lane >> 3;
            const uint2 sz = *reinterpret_cast<const uint2 *>(&stage.scale[c % kStages][2 * pair]);
            const float s_a = bf16_lo(sz.x), z_a = fmaf(8.0f, s_a, bf16_hi(sz.x));
            const float s_b = bf16_lo(sz.y), z_b = fmaf(8.0f, s_b, bf16_hi(sz.y));
            bool changed = false;
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                const int r = min(4 * i + sub, rows - 1);
                const uint2 d4 = *reinterpret_cast<const uint2 *>(&stage.dist[i][(16 * c + 2 * pair) % kQueue]);
                const uint32_t h_a = __byte_perm(d4.x, 0u, 0x4440 | sub), h_b = __byte_perm(d4.y, 0u, 0x4440 | sub);
                const float p_a = sh.p[r][h_a], p_b = sh.p[r][h_b];
                const float w_a = h_a == kUnseen ? 0.0f : p_a * s_a, w_b = h_b == kUnseen ? 0.0f : p_b * s_b;
                zacc[i] = zkeep[i] + ((h_a == kUnseen ? 0.0f : p_a * z_a) + (h_b == kUnseen ? 0.0f : p_b * z_b));
                // the chunk's largest weight, and not the largest that its scales allow: a key
                // of a huge scale and no weight would take the others' bits (NaN is no number
                // to scale by)
                float most = fmaxf(fabsf(w_a), fabsf(w_b));
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(kFullMask, most, o));
                // 2^12 <= most 2^(12 - e) < 2^13, with e >= -115
                const int e = max((int)(__float_as_uint(most) >> 23) - 127, -115);
                const float fit = most > 0.0f ? __uint_as_float((uint32_t)(12 - e + 127) << 23) : kMostScale;
                shrink[i] = 1.0f;
                if (most * scale[i] > kMostWeight) {
                    shrink[i] = fit / scale[i];
                    scale[i] = fit;
                    changed = true;
                }
                v_a[i] = w_a * scale[i];
                v_b[i] = w_b * scale[i];
            }
            return __any_sync(kFullMask, changed);
        };
        // Weights p s of chunk c, keys 2 (lane % 8) and the next, of every fourth
        // row, times the row's scale, as two fp16 terms.  True where a scale had
        // to come down: what was summed before is then to be shrunk.
        auto weigh = [&](int c) -> bool {
            const int pair = lane & 7, sub = lane >> 3;
            // row x of A and keys 2 pair, 2 pair + 1: a word of lane (x % 8, pair / 2)
            uint32_t *const terms = reinterpret_cast<uint32_t *>(stage.terms[c & 1]) + 16 * sub +
                                    4 * (pair >> 1) + 2 * (pair & 1);
            const uint2 sz = *reinterpret_cast<const uint2 *>(&stage.scale[c % kStages][2 * pair]);
            const float s_a = bf16_lo(sz.x), z_a = fmaf(8.0f, s_a, bf16_hi(sz.x));
            const float s_b = bf16_lo(sz.y), z_b = fmaf(8.0f, s_b, bf16_hi(sz.y));
            // a NaN scale must not meet the weight 0 of a row that drops the key
            bool odd = s_a != s_a || s_b != s_b;
            float v_a[RW], v_b[RW], zkeep[RW];
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                const int r = min(4 * i + sub, rows - 1);
                const uint2 d4 = *reinterpret_cast<const uint2 *>(&stage.dist[i][(16 * c + 2 * pair) % kQueue]);
                const uint32_t h_a = __byte_perm(d4.x, 0u, 0x4440 | sub), h_b = __byte_perm(d4.y, 0u, 0x4440 | sub);
                const float p_a = sh.p[r][h_a], p_b = sh.p[r][h_b];
                v_a[i] = p_a * scale[i] * s_a;
                v_b[i] = p_b * scale[i] * s_b;
                zkeep[i] = zacc[i];
                zacc[i] = fmaf(p_a, z_a, fmaf(p_b, z_b, zacc[i]));
                odd = odd || fmaxf(fabsf(v_a[i]), fabsf(v_b[i])) > kMostWeight;   // s of either sign
            }
            bool changed = false;
            if (__builtin_expect(__any_sync(kFullMask, odd), 0)) changed = reweigh(c, v_a, v_b, zkeep);
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                if (4 * i + sub >= rows) continue;
                const uint32_t hi = to_f16(v_a[i], v_b[i]);
                const float2 back = from_f16(hi);
                terms[64 * i] = hi;
                terms[64 * i + 1] = to_f16(v_a[i] - back.x, v_b[i] - back.y);
            }
            return changed;
        };
        auto fill = [&](int chunks) {
            while (queued < 16 * chunks && k0 < we) look();
        };
#pragma unroll 1
        for (int c = 0; c < kStages - 1; ++c) {
            fill(c + 1);
            __syncwarp();
            issue(c);
        }
        asm volatile("cp.async.wait_group %0;" :: "n"(kStages - 2) : "memory");
        __syncwarp();
        // (in the first segment nothing was summed before: what it returns does not matter)
        if (queued > 0 && weigh(0) && kLong) shrink_sums();
        // Step c issues the copies of chunk c + 3, weighs chunk c + 1 and
        // multiplies chunk c: the last two are independent, and one warp barrier
        // stands between a step's writes and the next step's reads.
        for (int c = 0; 16 * c < queued; ++c) {
            fill(c + kStages);
            asm volatile("cp.async.wait_group %0;" :: "n"(kStages - 3) : "memory");
            __syncwarp();
            issue(c + kStages - 1);
            const int ring = c % kStages;
            // this lane's four keys are 4 t4 .. 4 t4 + 3 and stand for columns
            // 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9 of A; its codes of a key are
            // elements g D/8 on
            uint32_t code[4][kCodeWords];
            const uint4 af = stage.terms[c & 1][g][t4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const unsigned char *from = stage.codes[ring] + (4 * t4 + e) * Stage::kStride + g * (D / 16);
                if constexpr (kCodeWords == 1) {
                    code[e][0] = *reinterpret_cast<const uint32_t *>(from);
                } else {
                    const uint2 u = *reinterpret_cast<const uint2 *>(from);
                    code[e][0] = u.x; code[e][1] = u.y;
                }
            }
            const bool smaller = 16 * (c + 1) < queued && weigh(c + 1);
#pragma unroll
            for (int w = 0; w < kCodeWords; ++w)
#pragma unroll
                for (int byte = 0; byte < 4; ++byte) {
                    const uint32_t sel = 0x4400 + 0x1111 * byte;       // that byte of both keys
                    const uint32_t x0 = __byte_perm(code[0][w], code[1][w], sel);
                    const uint32_t x1 = __byte_perm(code[2][w], code[3][w], sel);
                    mma_f16(acc[8 * w + 2 * byte], af, codes_low(x0, raised), codes_low(x1, raised));
                    mma_f16(acc[8 * w + 2 * byte + 1], af, codes_high(x0, raised), codes_high(x1, raised));
                }
            if (__builtin_expect(smaller, 0)) shrink_sums();       // the next chunk's scale
        }
        __syncwarp();
    }

    // a row's p z: eight lanes hold its parts
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) zacc[i] += __shfl_xor_sync(kFullMask, zacc[i], o);
    constexpr int kStride = kSumStride<D>;
    float *const sums = reinterpret_cast<float *>(attn_smem);
    const float unscale = 1.0f / of_row_g(scale);          // powers of two: exact
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int n = 2 * t4 + e % 2;
        if (g >= RM) continue;
        float *to = sums + (warp * 16 + g + 8 * (e / 2)) * kStride + n * kTiles;
#pragma unroll
        for (int i = 0; i < kTiles; i += 4)
            *reinterpret_cast<float4 *>(to + ((i / 4) ^ sum_swizzle<D>(n)) * 4) =
                make_float4(acc[i][e] * unscale, acc[i + 1][e] * unscale, acc[i + 2][e] * unscale,
                            acc[i + 3][e] * unscale);
    }
#pragma unroll
    for (int i = 0; i < RW; ++i)
        if ((lane & 7) == 0 && 4 * i + (lane >> 3) < rows) sh.zsum[warp][4 * i + (lane >> 3)] = zacc[i];
    __syncthreads();
    for (int e = tid; e < rows * D; e += kThreads) {
        const int r = e / D, k = e % D, n = k / kTiles, i = k % kTiles;
        const float *from = sums + r * kStride + n * kTiles + ((i / 4) ^ sum_swizzle<D>(n)) * 4 + i % 4;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w, from += 16 * kStride)
            sum += (from[8 * kStride] + sh.zsum[w][r]) + from[0];
        if (C > 1) sh.part[r][k] = sum;
        else a.out[q_row(r) * D + k] = sum;
    }
    if (C > 1) {
        cluster.sync();
        for (int e = rank * kThreads + tid; e < rows * D; e += C * kThreads) {
            const int r = e / D, k = e % D;
            float sum = 0.0f;
            for (int o = 0; o < C; ++o) sum += *cluster.map_shared_rank(&sh.part[r][k], o);
            a.out[q_row(r) * D + k] = sum;
        }
        cluster.sync();                       // the others have read this CTA's part
    }
}

}  // namespace had
