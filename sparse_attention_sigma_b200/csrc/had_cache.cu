// had_cache.cu -- the decoder cache's part of the C ABI of include/had.h:
// argument checks and kernel launches.
#include <climits>
#include <cstdint>
#include <cuda_runtime.h>

#include "had.h"
#include "had_cache.cuh"
#include "had_cache_attn.cuh"
#include "had_cache_pages.cuh"

namespace {

using had::Books;
using had::CacheTokens;
using had::CacheView;

constexpr int kMaxSmem = 227 * 1024;   // dynamic shared memory a CTA may have

bool aligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// A required array: there, and aligned.
bool good(const void *p, size_t to) { return p && aligned(p, to); }

had_status_t launched()
{
    return cudaGetLastError() == cudaSuccess ? HAD_OK : HAD_ERR_CUDA;
}

// A call that failed: its error is not left for the caller's next check.
had_status_t failed()
{
    cudaGetLastError();
    return HAD_ERR_CUDA;
}

bool good_page(int page)
{
    return page == 16 || page == 32 || page == 64 || page == 128 || page == 256;
}

int log2_of(int page)
{
    int l = 0;
    while ((1 << l) < page) ++l;
    return l;
}

had_status_t check_cache(const had_cache_t *c, CacheView *view)
{
    if (!c || c->pages < 1 || c->heads < 1 || c->d < 1) return HAD_ERR_INVALID_ARG;
    if (c->d != 64 && c->d != 128) return HAD_ERR_UNSUPPORTED;
    if (!good_page(c->page)) return HAD_ERR_UNSUPPORTED;
    // a (page, head, slot) row has a 32-bit index, and 2^32 - 1 stands for none
    if ((long long)c->pages * c->heads >= (1LL << 32) / c->page) return HAD_ERR_UNSUPPORTED;
    if (!good(c->kbits, 16) || !good(c->vcodes, 16) || !good(c->vscale, 16))
        return HAD_ERR_INVALID_ARG;
    view->kbits = c->kbits;
    view->vcodes = c->vcodes;
    view->vscale = static_cast<uint32_t *>(c->vscale);
    view->pages = c->pages;
    view->heads = c->heads;
    view->page_log = log2_of(c->page);
    return HAD_OK;
}

had_status_t check_table(const int32_t *table, int rows, int max_pages, int page)
{
    if (rows < 1 || max_pages < 1 || !good(table, 4)) return HAD_ERR_INVALID_ARG;
    // positions, and those of a few hundred keys behind the last, are ints
    return (long long)max_pages * page > INT_MAX - 65536 ? HAD_ERR_UNSUPPORTED : HAD_OK;
}

// The books of the page operators; `page` of 1 where a call has none.
had_status_t check_books(int32_t *table, const int32_t *lens, int32_t *refs, int S, int max_pages,
                         int pages, int page, Books *books)
{
    if (pages < 1 || !good(lens, 4) || !good(refs, 4)) return HAD_ERR_INVALID_ARG;
    if (page != 1 && !good_page(page)) return HAD_ERR_UNSUPPORTED;
    if (pages > INT_MAX - 65536) return HAD_ERR_UNSUPPORTED;     // a CTA's step past the last is an int
    const had_status_t s = check_table(table, S, max_pages, page);
    *books = Books{table, const_cast<int32_t *>(lens), refs, S, max_pages, pages, log2_of(page)};
    return s;
}

// A launch in clusters of `ctas` CTAs.  `most_smem`: the most that any launch of
// this kernel takes; the limit is set to that and never to less, since host
// threads that launch it at once share it.
template <typename... Params, typename... Args>
had_status_t launch_clusters(void (*kernel)(Params...), unsigned grid, unsigned ctas,
                             unsigned threads, size_t smem, size_t most_smem, cudaStream_t st,
                             Args... args)
{
    // 48 KB, the kernel's own variables included, need no attribute.  Set on
    // every call: it belongs to the current device.
    if (smem > 24 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)most_smem) != cudaSuccess)
        return failed();
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {ctas, 1, 1};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
    return e == cudaSuccess ? launched() : failed();
}

// A launch of one cluster of the page operators.
template <typename... Params, typename... Args>
had_status_t launch_cluster(void (*kernel)(Params...), size_t smem, size_t most_smem,
                            cudaStream_t st, Args... args)
{
    return launch_clusters(kernel, had::kBookCtas, had::kBookCtas, had::kBookThreads, smem,
                           most_smem, st, args...);
}

// Keys that a CTA holds at once at most: 20 KB of distances, so that four CTAs
// (three at d 128 with eight rows) share an SM.
template <int RW>
constexpr int kMostKeys = 20 * 1024 / (4 * RW) / 128 * 128;

template <int D, int RW, bool kLong>
had_status_t launch_attention_plan(const had::CacheAttnArgs &a, long long tiles,
                                   had::CacheAttnPlan plan, long long per, cudaStream_t st)
{
    constexpr int kThreads = had::kCacheAttnThreads;
    plan.cap = (int)((per + kThreads - 1) / kThreads * kThreads);
    if (tiles * plan.ctas > INT_MAX) return HAD_ERR_UNSUPPORTED;
    plan.by_tiles = had::divisor((unsigned)plan.tiles);
    plan.by_heads = had::divisor((unsigned)a.c.heads);
    plan.by_group = had::divisor((unsigned)(a.Hq / a.c.heads));
    return launch_clusters(had::cache_attn_kernel<D, RW, kLong>, (unsigned)(tiles * plan.ctas),
                           (unsigned)plan.ctas, kThreads,
                           had::cache_attn_smem_bytes<D, RW>(plan.cap),
                           had::cache_attn_smem_bytes<D, RW>(kMostKeys<RW>), st, a, plan);
}

template <int D, int RW>
had_status_t launch_attention_tile(const had::CacheAttnArgs &a, int B, int max_len, cudaStream_t st)
{
    const long long rows = (long long)(a.Hq / a.c.heads) * a.T;      // per key-value head
    had::CacheAttnPlan plan{};
    plan.tiles = (int)((rows + 4 * RW - 1) / (4 * RW));
    plan.R = (int)((rows + plan.tiles - 1) / plan.tiles);
    plan.tiles = (int)((rows + plan.R - 1) / plan.R);
    plan.ctas = 1;
    // the most keys a tile may see: the device alone knows the lengths
    long long keys = (long long)a.max_pages << a.c.page_log;
    if (a.window > 0) {
        const long long seen = (long long)a.window + a.sinks + plan.R;
        keys = seen < keys ? seen : keys;
    }
    const long long tiles = (long long)B * a.c.heads * plan.tiles;
    constexpr long long most = kMostKeys<RW>;
    // CTAs until four per SM are busy, each with 512 keys or more; the device uses
    // fewer for a tile that has fewer keys.  Measured with 1, 2, 4 and 8: 64 tiles
    // of 4 k keys 38, 23, 15.0, 15.2 us; 128 of 16 k 211, 129, 67, 73 us; 256 of
    // 1028 22.5, 21.5, 31, 58 us; one of 128 keys 6.4, 7.7, 7.4, 8.0 us.  More
    // CTAs, until their memory holds a tile's keys whole, only for as many keys as
    // the caller says there are: keys that do not fit are gone through twice (1024
    // tiles of 16 k keys 620 us instead of 426), but a table is often wider than
    // its sequences, and a cluster keeps its places until its last CTA is done (512
    // tiles of 4 k keys in a table for 128 k: 71 us, with 4 CTAs 94, with 8 149 us).
    const long long expected = max_len < keys ? max_len : keys;
    while (plan.ctas < had::kMaxCtas &&
           (expected > most * plan.ctas ||
            (tiles * plan.ctas * 2 <= 4 * 148 && keys > 512LL * plan.ctas)))
        plan.ctas *= 2;
    const long long per = (keys + plan.ctas - 1) / plan.ctas;
    return per <= most ? launch_attention_plan<D, RW, false>(a, tiles, plan, per, st)
                       : launch_attention_plan<D, RW, true>(a, tiles, plan, most, st);
}

// Tiles of 8 rows once clusters of four CTAs on them put three on every SM, of 4
// rows else.  A tile of 8 unpacks a kept key's codes for twice the rows, but
// fewer tiles split a decode's keys less finely.  Measured, 4 rows against 8, d 64:
// 4 x 512 queries under a window of 512 150, 125 us; 4 x 256 dense ones 100,
// 68; 16 decodes of 4 k tokens, 8 query heads to a key head, 16.8, 20 us;
// d 128: 91, 89; 74, 55; 20, 27 us.
template <int D>
had_status_t launch_attention(const had::CacheAttnArgs &a, int B, int max_len, cudaStream_t st)
{
    const long long rows = (long long)(a.Hq / a.c.heads) * a.T;
    if (rows > 4 && (rows + 7) / 8 * B * a.c.heads * 4 >= 3 * 148)
        return launch_attention_tile<D, 2>(a, B, max_len, st);
    return launch_attention_tile<D, 1>(a, B, max_len, st);
}

unsigned grid_for(long long items, int per_block)
{
    const long long blocks = (items + per_block - 1) / per_block, cap = 148LL * 8;
    return (unsigned)(blocks < cap ? blocks : cap);
}

template <typename T>
void launch_append(const void *K, const void *V, const float *sigma, const CacheView &c, int d,
                   const CacheTokens &k, unsigned grid, int32_t *status, cudaStream_t st)
{
    const auto *key = static_cast<const T *>(K), *value = static_cast<const T *>(V);
    if (d == 64)
        had::cache_append_kernel<T, 64><<<grid, 256, 0, st>>>(key, value, sigma, c, k, status);
    else
        had::cache_append_kernel<T, 128><<<grid, 256, 0, st>>>(key, value, sigma, c, k, status);
}

had_status_t check_rows(int B, int heads, int T)
{
    if (B < 1 || T < 1) return HAD_ERR_INVALID_ARG;
    const long long bh = (long long)B * heads;
    return bh > INT_MAX || bh * T > INT_MAX ? HAD_ERR_UNSUPPORTED : HAD_OK;
}

// Rows (b, head, token) of an append or a read, and the grid that has `lanes`
// threads for `at_once` of them.
CacheTokens tokens_of(const int32_t *table, int max_pages, const int32_t *start,
                      const int32_t *counts, int B, int heads, int T, int lanes, int at_once, unsigned *grid)
{
    const unsigned rows = (unsigned)B * heads * T, per = 256 / lanes * at_once;
    *grid = (rows + per - 1) / per;
    return CacheTokens{table, start, counts, max_pages, T, rows, had::divisor(T),
                       had::divisor(heads)};
}

bool finite_nonneg(float x) { return x >= 0.0f && x <= 3.4028234e38f; }

}  // namespace

extern "C" {

had_status_t had_cache_append(const void *K, const void *V, had_dtype_t dt, const float *sigma_k,
                              const had_cache_t *cache, const int32_t *table, int max_pages,
                              const int32_t *start, const int32_t *counts, int B, int T,
                              int32_t *dev_status, cudaStream_t stream)
{
    CacheView c;
    had_status_t s = check_cache(cache, &c);
    if (s == HAD_OK) s = check_rows(B, c.heads, T);
    if (s == HAD_OK) s = check_table(table, B, max_pages, cache->page);
    if (s != HAD_OK) return s;
    if (dt != HAD_BF16 && dt != HAD_F32) return HAD_ERR_INVALID_ARG;
    if (!good(K, 16) || !good(V, 16) || !good(sigma_k, 4) || !good(start, 4) ||
        !aligned(counts, 4) || !aligned(dev_status, 4))
        return HAD_ERR_INVALID_ARG;
    unsigned grid;
    const CacheTokens k = tokens_of(table, max_pages, start, counts, B, c.heads, T,
                                    had::kCacheLanes, had::kCacheRows, &grid);
    if (dt == HAD_BF16)
        launch_append<__nv_bfloat16>(K, V, sigma_k, c, cache->d, k, grid, dev_status, stream);
    else
        launch_append<float>(K, V, sigma_k, c, cache->d, k, grid, dev_status, stream);
    return launched();
}

had_status_t had_cache_read(const had_cache_t *cache, const int32_t *table, int max_pages,
                            const int32_t *start, const int32_t *counts, int B, int T,
                            uint32_t *bits, float *values, int32_t *dev_status,
                            cudaStream_t stream)
{
    CacheView c;
    had_status_t s = check_cache(cache, &c);
    if (s == HAD_OK) s = check_rows(B, c.heads, T);
    if (s == HAD_OK) s = check_table(table, B, max_pages, cache->page);
    if (s != HAD_OK) return s;
    if (!good(start, 4) || !aligned(counts, 4) || !aligned(bits, 16) || !aligned(values, 16) ||
        !aligned(dev_status, 4))
        return HAD_ERR_INVALID_ARG;
    if (!bits && !values) return HAD_ERR_INVALID_ARG;
    unsigned grid;
    const CacheTokens k = tokens_of(table, max_pages, start, counts, B, c.heads, T,
                                    had::kReadLanes, had::kReadRows, &grid);
    if (cache->d == 64)
        had::cache_read_kernel<64><<<grid, 256, 0, stream>>>(c, k, bits, values, dev_status);
    else
        had::cache_read_kernel<128><<<grid, 256, 0, stream>>>(c, k, bits, values, dev_status);
    return launched();
}

had_status_t had_cache_attention(const void *Q, had_dtype_t dt, const float *sigma_q,
                                 const had_cache_t *cache, const int32_t *table, int max_pages,
                                 const int32_t *lens, const int32_t *counts, int B, int Hq, int T,
                                 int N, float tau, int window, int sinks, int max_len, float *out,
                                 int32_t *dev_status, cudaStream_t stream)
{
    CacheView c;
    had_status_t s = check_cache(cache, &c);
    if (s == HAD_OK && Hq < 1) s = HAD_ERR_INVALID_ARG;
    if (s == HAD_OK) s = check_rows(B, Hq, T);
    if (s == HAD_OK) s = check_table(table, B, max_pages, cache->page);
    if (s != HAD_OK) return s;
    if (Hq % c.heads != 0 || N < 1 || window < 0 || sinks < 0 || max_len < 0 ||
        !finite_nonneg(tau))
        return HAD_ERR_INVALID_ARG;
    if (dt != HAD_BF16 && dt != HAD_F32) return HAD_ERR_INVALID_ARG;
    if (!good(Q, 16) || !good(out, 16) || !good(sigma_q, 4) || !good(lens, 4) ||
        !aligned(counts, 4) || !aligned(dev_status, 4))
        return HAD_ERR_INVALID_ARG;
    const had::CacheAttnArgs a{Q, dt == HAD_BF16, sigma_q, c, table, lens, counts, max_pages, Hq, T, N, window,
                               sinks, tau, out, dev_status};
    return cache->d == 64 ? launch_attention<64>(a, B, max_len, stream)
                          : launch_attention<128>(a, B, max_len, stream);
}

had_status_t had_cache_fork(int32_t *table, int32_t *lens, int32_t *refs, int S, int max_pages,
                            int pages, int page, const int32_t *src, const int32_t *dst, int n,
                            int32_t *dev_status, cudaStream_t stream)
{
    Books k;
    if (page == 1) return HAD_ERR_UNSUPPORTED;
    const had_status_t s = check_books(table, lens, refs, S, max_pages, pages, page, &k);
    if (s != HAD_OK) return s;
    if (S > had::kMaxSeqs) return HAD_ERR_UNSUPPORTED;
    if (n < 0 || n > S) return HAD_ERR_INVALID_ARG;
    if (n == 0) return HAD_OK;
    if (!good(src, 4) || !good(dst, 4) || !aligned(dev_status, 4)) return HAD_ERR_INVALID_ARG;
    // whole 128-byte lines of a row per tile while shared memory holds them
    int tile = 32;
    while (tile > 1 && had::fork_smem_bytes(n, S, tile) > (size_t)kMaxSmem) --tile;
    return launch_cluster(had::cache_fork_kernel, had::fork_smem_bytes(n, S, tile), kMaxSmem, stream,
                          k, src, dst, n, tile, dev_status);
}

had_status_t had_cache_reserve(int32_t *table, const int32_t *lens, int32_t *refs, int S,
                               int max_pages, int pages, int page, const int32_t *grow,
                               int32_t *src, int32_t *dst, int32_t *dev_status,
                               cudaStream_t stream)
{
    Books k;
    if (page == 1) return HAD_ERR_UNSUPPORTED;
    const had_status_t s = check_books(table, lens, refs, S, max_pages, pages, page, &k);
    if (s != HAD_OK) return s;
    if (S > had::kMaxSeqs) return HAD_ERR_UNSUPPORTED;
    if (!good(grow, 4) || !good(src, 4) || !good(dst, 4) || !aligned(dev_status, 4))
        return HAD_ERR_INVALID_ARG;
    return launch_cluster(had::cache_reserve_kernel, had::reserve_smem_bytes(S),
                          had::reserve_smem_bytes(had::kMaxSeqs), stream, k, grow, src, dst,
                          dev_status);
}

had_status_t had_cache_free(int32_t *table, int32_t *lens, int32_t *refs, int S, int max_pages,
                            int pages, const int32_t *seqs, int n, int32_t *dev_status,
                            cudaStream_t stream)
{
    Books k;
    const had_status_t s = check_books(table, lens, refs, S, max_pages, pages, 1, &k);
    if (s != HAD_OK) return s;
    if (n < 0) return HAD_ERR_INVALID_ARG;
    if (n == 0) return HAD_OK;
    if (!good(seqs, 4) || !aligned(dev_status, 4)) return HAD_ERR_INVALID_ARG;
    had::cache_free_kernel<<<grid_for((long long)n * max_pages, 256), 256, 0, stream>>>(
        k, seqs, n, dev_status);
    return launched();
}

had_status_t had_cache_evict(int32_t *table, const int32_t *lens, int32_t *refs, int S,
                             int max_pages, int pages, int page, int window, int sinks,
                             int32_t *dev_status, cudaStream_t stream)
{
    Books k;
    if (page == 1) return HAD_ERR_UNSUPPORTED;
    const had_status_t s = check_books(table, lens, refs, S, max_pages, pages, page, &k);
    if (s != HAD_OK) return s;
    if (window < 1 || sinks < 0 || !aligned(dev_status, 4)) return HAD_ERR_INVALID_ARG;
    had::cache_evict_kernel<<<grid_for((long long)S * max_pages, 256), 256, 0, stream>>>(
        k, window, sinks, dev_status);
    return launched();
}

had_status_t had_cache_compact(int32_t *table, int32_t *refs, int S, int max_pages, int pages,
                               int32_t *src, int32_t *dst, int32_t *live, int32_t *dev_status,
                               cudaStream_t stream)
{
    Books k;
    const had_status_t s = check_books(table, refs, refs, S, max_pages, pages, 1, &k);
    if (s != HAD_OK) return s;
    if (!good(src, 4) || !good(dst, 4) || !good(live, 4) || !aligned(dev_status, 4))
        return HAD_ERR_INVALID_ARG;
    return launch_cluster(had::cache_compact_kernel, 0, 0, stream, k, src, dst, live, dev_status);
}

had_status_t had_cache_copy_pages(const had_cache_t *cache, const int32_t *src,
                                  const int32_t *dst, int n, int32_t *dev_status,
                                  cudaStream_t stream)
{
    CacheView c;
    const had_status_t s = check_cache(cache, &c);
    if (s != HAD_OK) return s;
    if (n < 0) return HAD_ERR_INVALID_ARG;
    if (n == 0) return HAD_OK;
    if (!good(src, 4) || !good(dst, 4) || !aligned(dev_status, 4)) return HAD_ERR_INVALID_ARG;
    const long long rows = (long long)c.heads * cache->page, d = cache->d;
    const had::CopyWords words{rows * d / 32, rows * d / 128, rows / 4};
    had::cache_copy_kernel<<<dim3(had::kCopyParts, n < 512 ? n : 512), 256, 0, stream>>>(
        c, words, src, dst, n, dev_status);
    return launched();
}

}  // extern "C"
