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
// of the softmax; a second pass over the keys takes the values.
#pragma once
#include "had_cache.cuh"

namespace had {

struct CacheAttnArgs {
    const void *Q;
    const float *sigma;
    CacheView c;
    const int32_t *table, *lens, *counts;
    int max_pages, Hq, T, N, window, sinks;
    float tau;
    float *out;
    int32_t *status;
};

constexpr int kCacheAttnThreads = 256;

// Visible range of a row: keys [0, sinks) and [lo, pos], pos = -1 for none.
struct RowRange {
    int sinks, lo, pos;
};

__device__ __forceinline__ RowRange row_range(const CacheAttnArgs &a, int len, int count, int t)
{
    RowRange r;
    r.pos = t < count ? len - count + t : -1;
    if (r.pos < 0) r.pos = -1;
    r.lo = a.window > 0 ? max(0, r.pos - a.window + 1) : 0;
    r.sinks = min(a.sinks, r.lo);
    return r;
}

// One CTA per row: distances and histogram, threshold, then the kept tokens
// 256 at a time.
template <typename T, int D>
__global__ void __launch_bounds__(kCacheAttnThreads)
cache_attn_row_kernel(CacheAttnArgs a)
{
    constexpr int DW = D / 32;
    constexpr int kWarps = kCacheAttnThreads / 32;
    constexpr int kParts = kCacheAttnThreads / (D / 2);
    __shared__ uint32_t qbits[DW];
    __shared__ int hist[D + 1];
    __shared__ float weight[D + 1];
    __shared__ int level, quota, warp_ties[kWarps], warp_kept[kWarps];
    __shared__ long long kept_row[kCacheAttnThreads];
    __shared__ float kept_p[kCacheAttnThreads];
    __shared__ float sums[kParts][D];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x;
    const int t = (int)(row % a.T);
    const int hq = (int)(row / a.T % a.Hq), b = (int)(row / a.T / a.Hq);
    const int h = hq / (a.Hq / a.c.heads);
    const int32_t *table = a.table + (long long)b * a.max_pages;
    int len = a.lens[b], count = a.counts ? a.counts[b] : a.T;
    if (len < 0 || len > (long long)a.max_pages << a.c.page_log || count < 0 || count > a.T) {
        if (tid == 0) flag(a.status, HAD_ERR_INVALID_ARG);
        len = count = 0;
    }
    const RowRange rr = row_range(a, len, count, t);
    const int total = rr.pos < 0 ? 0 : rr.sinks + rr.pos + 1 - rr.lo;

    const SignRule rule = sign_rule(a.sigma[hq]);
    if (tid < D) {
        if (rule.bad && tid == 0) flag(a.status, HAD_ERR_BAD_SIGMA);
        const float x = (float)static_cast<const T *>(a.Q)[row * D + tid];
        const uint32_t w = __ballot_sync(kFullMask, negative_bit(x, rule));
        if (lane == 0) qbits[warp] = w;
    }
    for (int l = tid; l <= D; l += kCacheAttnThreads) hist[l] = 0;
    __syncthreads();

    // row of key u of the visible ones, or -1 where the table holds no page
    auto place = [&](int u) -> long long {
        const int j = u < rr.sinks ? u : u - rr.sinks + rr.lo;
        const int page = table[j >> a.c.page_log];
        if (page < 0 || page >= a.c.pages) return -1;
        return cache_row(a.c, page, h, j & ((1 << a.c.page_log) - 1));
    };
    auto distance = [&](long long at) -> int {
        int n = 0;
#pragma unroll
        for (int w = 0; w < DW; ++w) n += __popc(a.c.kbits[at * DW + w] ^ qbits[w]);
        return n;
    };
    for (int u = tid; u < total; u += kCacheAttnThreads) {
        const long long at = place(u);
        if (at < 0)
            flag(a.status, HAD_ERR_INVALID_ARG);
        else
            atomicAdd(&hist[distance(at)], 1);
    }
    __syncthreads();
    if (tid == 0) {
        int first = -1, seen = 0, l = 0;
        float z = 0.0f;
        level = -1;
        quota = 0;
        for (; l <= D && seen < a.N; ++l) {
            weight[l] = 0.0f;
            if (hist[l] == 0) continue;
            if (first < 0) first = l;
            const int n = min(hist[l], a.N - seen);
            weight[l] = expf(a.tau * (float)(2 * (first - l)));
            z += (float)n * weight[l];
            seen += n;
            level = l;
            quota = n;
        }
        for (int k = 0; k <= level; ++k) weight[k] /= z;
    }
    __syncthreads();

    const int t_level = level;
    int t_quota = quota;
    const int pair = tid % (D / 2), part = tid / (D / 2);
    float acc0 = 0.0f, acc1 = 0.0f;
    for (int u0 = 0; u0 < total; u0 += kCacheAttnThreads) {
        const long long at = u0 + tid < total ? place(u0 + tid) : -1;
        const int dist = at >= 0 ? distance(at) : D + 1;
        const unsigned ties = __ballot_sync(kFullMask, dist == t_level);
        if (lane == 0) warp_ties[warp] = __popc(ties);
        __syncthreads();
        int before = __popc(ties & ((1u << lane) - 1)), all = 0;
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? warp_ties[w] : 0;
            all += warp_ties[w];
        }
        const bool keep = dist < t_level || (dist == t_level && before < t_quota);
        t_quota -= min(all, t_quota);
        const unsigned kept = __ballot_sync(kFullMask, keep);
        if (lane == 0) warp_kept[warp] = __popc(kept);
        __syncthreads();
        int slot = __popc(kept & ((1u << lane) - 1)), n = 0;
        for (int w = 0; w < kWarps; ++w) {
            slot += w < warp ? warp_kept[w] : 0;
            n += warp_kept[w];
        }
        if (keep) {
            kept_row[slot] = at;
            kept_p[slot] = weight[dist];
        }
        __syncthreads();
        for (int k = part; k < n; k += kParts) {
            const long long r = kept_row[k];
            const uint32_t code = a.c.vcodes[r * (D / 2) + pair], sz = a.c.vscale[r];
            acc0 = fmaf(kept_p[k], fmaf((float)(code & 15u), bf16_lo(sz), bf16_hi(sz)), acc0);
            acc1 = fmaf(kept_p[k], fmaf((float)(code >> 4), bf16_lo(sz), bf16_hi(sz)), acc1);
        }
    }
    sums[part][2 * pair] = acc0;
    sums[part][2 * pair + 1] = acc1;
    __syncthreads();
    if (tid < D) {
        float o = sums[0][tid];
        for (int k = 1; k < kParts; ++k) o += sums[k][tid];
        a.out[row * D + tid] = o;
    }
}

}  // namespace had
