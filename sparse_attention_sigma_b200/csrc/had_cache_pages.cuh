// had_cache_pages.cuh -- the books of the decoder cache's pages: which
// sequence holds which page, how many hold it, and moving pages.
//
// table [S, max_pages] int32 lists the pages of every sequence (-1: none),
// lens [S] its tokens, refs [P] how many table entries name a page (0: free).
// The kernels that need the whole table or all of refs at once run as one
// cluster of CTAs: what the others have to know goes through distributed
// shared memory, and the cluster's barrier stands between the last read of
// the old books and the first write of the new ones.  These operators move a
// few hundred KB at most and are bound by the latency of a launch and of a
// few dependent loads, so one launch each is the point.
#pragma once
#include <cooperative_groups.h>

#include "had_cache.cuh"

namespace had {

namespace cg = cooperative_groups;

constexpr int kBookCtas = 8;           // CTAs of the cluster
constexpr int kBookThreads = 512;
constexpr int kBookWarps = kBookThreads / 32;
constexpr int kMaxSeqs = 8192;         // rows of a table: bounded by shared memory

struct Books {
    int32_t *table, *lens, *refs;
    int seqs, max_pages, pages, page_log;
};

// Sum over the CTA; every thread gets it.  `buf` holds one int per warp.
__device__ __forceinline__ int block_sum(int x, int *buf)
{
    x = __reduce_add_sync(kFullMask, x);
    __syncthreads();                       // buf may still be read from before
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    int s = 0;
    for (int w = 0; w < kBookWarps; ++w) s += buf[w];
    return s;
}

// Exclusive prefix over the CTA's threads; `all` gets the sum.
template <typename I>
__device__ __forceinline__ I block_prefix(I x, I *buf, I &all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    I in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const I y = __shfl_up_sync(kFullMask, in, o);
        if (lane >= o) in += y;
    }
    __syncthreads();
    if (lane == 31) buf[warp] = in;
    __syncthreads();
    I before = 0;
    all = 0;
    for (int w = 0; w < kBookWarps; ++w) {
        before += w < warp ? buf[w] : 0;
        all += buf[w];
    }
    return before + in - x;
}

__device__ __forceinline__ int pages_of(int tokens, int page_log)
{
    return (int)(((long long)tokens + (1 << page_log) - 1) >> page_log);
}

// Sequence dst[i] goes on as a copy of sequence src[i], for all i at once:
// its old pages are let go and it shares the pages of src[i]'s tokens.  CTA
// r of the cluster takes tiles of `tile` columns; a tile's old entries are all
// read before its first new one is written, and a source may be another
// pair's destination.  Nothing is changed where an index or a length is out of
// range or a destination is listed twice.
inline size_t fork_smem_bytes(int n, int seqs, int tile)
{
    return sizeof(int) * ((size_t)n * (tile + 1) + (seqs + 31) / 32);
}

__global__ void __launch_bounds__(kBookThreads)
cache_fork_kernel(Books k, const int32_t *__restrict__ src, const int32_t *__restrict__ dst,
                  int n, int tile, int32_t *status)
{
    extern __shared__ int fork_smem[];
    int *entry = fork_smem, *len = entry + n * tile;
    unsigned *seen = reinterpret_cast<unsigned *>(len + n);
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, rank = (int)cluster.block_rank();
    const int words = (k.seqs + 31) / 32;
    for (int w = tid; w < words; w += kBookThreads) seen[w] = 0u;
    __syncthreads();
    int bad = 0;
    for (int i = tid; i < n; i += kBookThreads) {
        const int s = src[i], d = dst[i];
        if (s < 0 || s >= k.seqs || d < 0 || d >= k.seqs) {
            bad = 1;
            continue;
        }
        if (atomicOr(&seen[d >> 5], 1u << (d & 31)) >> (d & 31) & 1u) bad = 1;
        len[i] = k.lens[s];
        if (len[i] < 0 || len[i] > (long long)k.max_pages << k.page_log) bad = 1;
    }
    bad = __syncthreads_or(bad);
    cluster.sync();                        // every CTA has the old lengths
    if (bad) {                             // the same in every CTA
        if (rank == 0 && tid == 0) flag(status, HAD_ERR_INVALID_ARG);
        return;
    }
    if (rank == 0)
        for (int i = tid; i < n; i += kBookThreads) k.lens[dst[i]] = len[i];
    for (int c0 = rank * tile; c0 < k.max_pages; c0 += kBookCtas * tile) {
        const int cols = min(tile, k.max_pages - c0);
        for (int e = tid; e < n * cols; e += kBookThreads) {
            const int i = e / cols, c = e - i * cols;
            int p = -1;
            if (c0 + c < pages_of(len[i], k.page_log))
                p = k.table[(long long)src[i] * k.max_pages + c0 + c];
            if (p >= k.pages) {
                flag(status, HAD_ERR_INVALID_ARG);
                p = -1;
            }
            if (p >= 0) atomicAdd(k.refs + p, 1);
            entry[i * tile + c] = p < 0 ? -1 : p;
        }
        __syncthreads();
        for (int e = tid; e < n * cols; e += kBookThreads) {
            const int i = e / cols, c = e - i * cols;
            int32_t *at = k.table + (long long)dst[i] * k.max_pages + c0 + c;
            const int old = *at;
            if (old >= 0 && old < k.pages)
                atomicSub(k.refs + old, 1);
            else if (old >= 0)
                flag(status, HAD_ERR_INVALID_ARG);
            *at = entry[i * tile + c];
        }
        __syncthreads();
    }
}

// Room for grow[s] more tokens of every sequence: fresh pages behind the ones
// it has, and a page of its own where its last, partly filled page is shared
// (that page's content is to be copied: src -> dst).  The free pages go out in
// ascending order to ascending (sequence, entry).  Of the growing sequences
// that share a last page the last one keeps it when nobody else holds it.
//
// Entries behind a length are kept, but for pages that another entry names as
// well (a length that went back after a fork leaves such): those are let go for
// fresh ones.  Missing entries are filled where they stand.
//
// Each CTA looks at an eighth of the sequences and at an eighth of refs; three
// cluster barriers pass on what the others need: the last pages, the numbers
// of wanted and of free pages, and that all have read the old books.  Rows whose
// wanted entries are not simply the last ones take two more: an owner first
// writes each such entry's number among the row's into the table, where the
// thread that has the page of that number finds it.  A page that is let go
// meanwhile carries kLetGo, so that it is seen as shared and not as free until
// all are done.
struct ReserveShared {
    long long wide[kBookWarps];
    int buf[kBookWarps];
    int free_pages, bad, uneven;
};

constexpr int kLetGo = 1 << 30;        // in refs, which stay far below

inline size_t reserve_smem_bytes(int seqs)
{
    return sizeof(int) * (4 * (size_t)seqs + 1);
}

__global__ void __launch_bounds__(kBookThreads)
cache_reserve_kernel(Books k, const int32_t *__restrict__ grow, int32_t *src, int32_t *dst,
                     int32_t *status)
{
    extern __shared__ int reserve_smem[];
    int *last = reserve_smem;              // [S] shared last page of a growing sequence, or -1
    int *first = last + k.seqs;            // [S] first entry that gets a fresh page, ~ of it in an uneven row
    int *need = first + k.seqs;            // [S] fresh pages wanted; the copy, if any, included
    int *upto = need + k.seqs;             // [S + 1] exclusive prefix of need
    __shared__ ReserveShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster.block_rank();
    const int s0 = (int)((long long)k.seqs * rank / kBookCtas);
    const int s1 = (int)((long long)k.seqs * (rank + 1) / kBookCtas);
    const int p0 = (int)((long long)k.pages * rank / kBookCtas);
    const int p1 = (int)((long long)k.pages * (rank + 1) / kBookCtas);
    const int page = 1 << k.page_log;

    // behind the length: a page that another entry names as well
    auto shared_behind = [&](int p) { return p < k.pages && k.refs[p] > 1; };

    // a warp per sequence
    int bad = 0, uneven = 0;
    for (int s = s0 + warp; s < s1; s += kBookWarps) {
        const int len = k.lens[s], g = grow[s];
        int shared_page = -1, from = 0, wanted = 0;
        const bool fits = len >= 0 && g >= 0 &&
                          (long long)len + g <= (long long)k.max_pages << k.page_log;
        if (!fits) {
            bad = 1;
        } else if (g > 0) {
            const int32_t *row = k.table + (long long)s * k.max_pages;
            const int have = pages_of(len, k.page_log), want = pages_of(len + g, k.page_log);
            if (len & (page - 1)) {
                const int p = row[have - 1];
                if (p < 0 || p >= k.pages)
                    bad = 1;
                else if (k.refs[p] > 1)
                    shared_page = p;
            }
            // entries held from an earlier call come first, as a rule, then those to be filled
            from = want;
            int odd = 0;
            for (int c0 = have; c0 < want; c0 += 32) {
                const int p = c0 + lane < want ? row[c0 + lane] : -1;
                if (p >= k.pages) bad = 1;
                const bool none = p < 0 && c0 + lane < want, swap = p >= 0 && shared_behind(p);
                const unsigned fill = __ballot_sync(kFullMask, none || swap);
                if (fill && from == want) from = c0 + __ffs(fill) - 1;
                wanted += __popc(fill);
                odd |= p >= 0 && (swap || c0 + lane > from);
            }
            if (__any_sync(kFullMask, odd)) {
                uneven = 1;
                from = ~from;
            }
        }
        if (lane == 0) {
            last[s] = shared_page;
            first[s] = from;
            need[s] = wanted;
        }
    }
    int n = 0;
#pragma unroll 4
    for (int p = p0 + tid; p < p1; p += kBookThreads) n += k.refs[p] == 0;
    n = block_sum(n, sh.buf);
    bad = __syncthreads_or(bad);
    uneven = __syncthreads_or(uneven);
    if (tid == 0) {
        sh.free_pages = n;
        sh.bad = bad;
        sh.uneven = uneven;
    }
    cluster.sync();
    for (int s = tid; s < k.seqs; s += kBookThreads) {
        // the CTA that looked at s: the smallest r with s < S (r + 1) / 8
        const int r = (int)(((long long)(s + 1) * kBookCtas - 1) / k.seqs);
        if (r != rank) last[s] = cluster.map_shared_rank(last, r)[s];
    }
    __syncthreads();
    for (int s = s0 + tid; s < s1; s += kBookThreads) {
        const int p = last[s];
        if (p < 0) continue;
        int earlier = 0;
        for (int o = 0; o < s; ++o) earlier += last[o] == p;
        // marked only after the barrier: others still read `last` of this CTA
        need[s] += k.refs[p] - earlier > 1 ? 1 << 30 : 0;
    }
    int free_pages = 0, before = 0;
    for (int r = 0; r < kBookCtas; ++r) {
        const ReserveShared *o = cluster.map_shared_rank(&sh, r);
        before += r < rank ? o->free_pages : 0;
        free_pages += o->free_pages;
        bad |= o->bad;
        uneven |= o->uneven;
    }
    cluster.sync();
    for (int s = tid; s < k.seqs; s += kBookThreads) {
        const int r = (int)(((long long)(s + 1) * kBookCtas - 1) / k.seqs);
        if (r != rank) {
            need[s] = cluster.map_shared_rank(need, r)[s];
            first[s] = cluster.map_shared_rank(first, r)[s];
        }
    }
    __syncthreads();
    cluster.sync();                        // nobody reads another CTA's arrays from here on
    // exclusive prefix of the wanted pages, a run of sequences per thread
    const int run = (k.seqs + kBookThreads - 1) / kBookThreads;
    const int r0 = min(k.seqs, tid * run), r1 = min(k.seqs, r0 + run);
    long long mine = 0;
    for (int s = r0; s < r1; ++s) {
        const bool copy = need[s] >> 30 & 1;
        need[s] = (need[s] & ~(1 << 30)) + copy;
        if (!copy) last[s] = -1;
        mine += need[s];
    }
    long long wanted = 0;
    long long at = block_prefix(mine, sh.wide, wanted);
    const bool refuse = bad || wanted > free_pages;
    const int total = refuse ? 0 : (int)wanted;
    for (int s = r0; s < r1; ++s) {
        upto[s] = refuse ? 0 : (int)at;
        at += need[s];
    }
    if (tid == 0) upto[k.seqs] = total;
    __syncthreads();
    if (refuse && rank == 0 && tid == 0)
        flag(status, bad ? HAD_ERR_INVALID_ARG : HAD_ERR_NO_PAGES);
    for (int s = s0 + tid; s < s1; s += kBookThreads) {
        const bool copy = !refuse && last[s] >= 0;
        src[s] = copy ? last[s] : -1;
        if (!copy) dst[s] = -1;
        if (copy) {
            if (uneven) atomicOr(k.refs + last[s], kLetGo);
            atomicSub(k.refs + last[s], 1);
        }
    }
    if (refuse) return;
    if (uneven) {                          // the same in every CTA
        for (int s = s0 + warp; s < s1; s += kBookWarps) {
            if (first[s] >= 0) continue;
            int32_t *row = k.table + (long long)s * k.max_pages;
            const int want = pages_of(k.lens[s] + grow[s], k.page_log);
            int nth = 0;
            for (int c0 = ~first[s]; c0 < want; c0 += 32) {
                const int c = c0 + lane, p = c < want ? row[c] : -1;
                const bool swap = p >= 0 && shared_behind(p);
                if (swap) {
                    atomicOr(k.refs + p, kLetGo);
                    atomicSub(k.refs + p, 1);
                }
                const bool fill = c < want && (p < 0 || swap);
                const unsigned fills = __ballot_sync(kFullMask, fill);
                if (fill) row[c] = -2 - nth - __popc(fills & ((1u << lane) - 1));
                nth += __popc(fills);
            }
        }
        cluster.sync();
    }
    // the free pages of this CTA's range to the entries of the same ranks
    for (int q0 = p0; q0 < p1 && before < total; q0 += kBookThreads) {
        const int p = q0 + tid;
        const bool is_free = p < p1 && k.refs[p] == 0;
        int all;
        const int i = before + block_prefix((int)is_free, sh.buf, all);
        before += all;
        if (!is_free || i >= total) continue;
        int lo = 0, hi = k.seqs;           // the sequence with upto[lo] <= i < upto[lo + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (upto[mid] <= i) lo = mid;
            else hi = mid;
        }
        const int nth = i - upto[lo];
        int32_t *row = k.table + (long long)lo * k.max_pages;
        const bool copy = last[lo] >= 0;
        if (copy && nth == 0) {
            row[pages_of(k.lens[lo], k.page_log) - 1] = p;
            dst[lo] = p;
        } else if (first[lo] >= 0) {
            row[first[lo] + nth - copy] = p;
        } else {
            int c = ~first[lo] + nth - copy;       // or behind it, by as many entries as are kept
            while (c < k.max_pages - 1 && row[c] != -2 - (nth - copy)) ++c;
            row[c] = p;
        }
        k.refs[p] = 1;
    }
    if (uneven) {
        cluster.sync();                    // nobody looks for free pages any more
        for (int p = p0 + tid; p < p1; p += kBookThreads)
            if (k.refs[p] > 0 && (k.refs[p] & kLetGo)) k.refs[p] &= ~kLetGo;
    }
}

// All entries of the listed sequences are let go and their lengths become 0.
// The exchange hands every entry to one thread only, so a sequence may be
// listed twice.
__global__ void __launch_bounds__(256)
cache_free_kernel(Books k, const int32_t *__restrict__ seqs, int n, int32_t *status)
{
    const long long total = (long long)n * k.max_pages;
    for (long long e = blockIdx.x * 256LL + threadIdx.x; e < total; e += gridDim.x * 256LL) {
        const int i = (int)(e / k.max_pages), c = (int)(e - (long long)i * k.max_pages);
        const int s = seqs[i];
        if (s < 0 || s >= k.seqs) {
            if (c == 0) flag(status, HAD_ERR_INVALID_ARG);
            continue;
        }
        const int p = atomicExch(k.table + (long long)s * k.max_pages + c, -1);
        if (p >= k.pages)
            flag(status, HAD_ERR_INVALID_ARG);
        else if (p >= 0)
            atomicSub(k.refs + p, 1);
        if (c == 0) k.lens[s] = 0;
    }
}

// Entries whose tokens no later query sees under the window are let go: those
// that hold only positions in [sinks, len - window).
__global__ void __launch_bounds__(256)
cache_evict_kernel(Books k, int window, int sinks, int32_t *status)
{
    const long long total = (long long)k.seqs * k.max_pages;
    for (long long e = blockIdx.x * 256LL + threadIdx.x; e < total; e += gridDim.x * 256LL) {
        const int s = (int)(e / k.max_pages), c = (int)(e - (long long)s * k.max_pages);
        const long long first = (long long)c << k.page_log;
        if (first < sinks || first + (1 << k.page_log) > (long long)k.lens[s] - window) continue;
        const int p = k.table[e];
        if (p < 0) continue;
        k.table[e] = -1;
        if (p >= k.pages)
            flag(status, HAD_ERR_INVALID_ARG);
        else
            atomicSub(k.refs + p, 1);
    }
}

// Closes the holes of a pool: with `live` pages in use, the k-th used page at
// or beyond `live` moves into the k-th free page below it.  Table and refs are
// changed here, src -> dst names the contents to be copied.
//
// Each CTA counts an eighth of refs, then the holes and the far pages of it,
// ranks them, and after the pairs are known in all CTAs moves refs and renames
// an eighth of the table; a page's new place is found by bisection, src being
// ascending.
struct CompactShared {
    int buf[kBookWarps];
    int used, holes, far;
};

__global__ void __launch_bounds__(kBookThreads)
cache_compact_kernel(Books k, int32_t *src, int32_t *dst, int32_t *live_out, int32_t *status)
{
    __shared__ CompactShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, rank = (int)cluster.block_rank();
    const int p0 = (int)((long long)k.pages * rank / kBookCtas);
    const int p1 = (int)((long long)k.pages * (rank + 1) / kBookCtas);
    int n = 0;
#pragma unroll 4
    for (int p = p0 + tid; p < p1; p += kBookThreads) n += k.refs[p] > 0;
    n = block_sum(n, sh.buf);
    if (tid == 0) sh.used = n;
    cluster.sync();
    int live = 0;
    for (int r = 0; r < kBookCtas; ++r) live += cluster.map_shared_rank(&sh, r)->used;
    int holes = 0, far = 0;
#pragma unroll 4
    for (int p = p0 + tid; p < p1; p += kBookThreads) {
        const bool used = k.refs[p] > 0;
        holes += p < live && !used;
        far += p >= live && used;
    }
    holes = block_sum(holes, sh.buf);
    far = block_sum(far, sh.buf);
    if (tid == 0) {
        sh.holes = holes;
        sh.far = far;
    }
    cluster.sync();
    int moves = 0, h0 = 0, f0 = 0;
    for (int r = 0; r < kBookCtas; ++r) {
        const CompactShared *o = cluster.map_shared_rank(&sh, r);
        moves += o->far;
        h0 += r < rank ? o->holes : 0;
        f0 += r < rank ? o->far : 0;
    }
    for (int q0 = p0; q0 < p1; q0 += kBookThreads) {
        const int p = q0 + tid;
        const bool used = p < p1 && k.refs[p] > 0;
        const bool hole = p < p1 && p < live && !used, is_far = p < p1 && p >= live && used;
        int all;
        const int hi = h0 + block_prefix((int)hole, sh.buf, all);
        h0 += all;
        const int fi = f0 + block_prefix((int)is_far, sh.buf, all);
        f0 += all;
        if (hole) dst[hi] = p;
        if (is_far) src[fi] = p;
        if (p < p1 && p >= moves) src[p] = dst[p] = -1;
    }
    if (rank == 0 && tid == 0) *live_out = live;
    cluster.sync();                        // the pairs are written, refs all read
    const int step = kBookCtas * kBookThreads;
    for (int i = rank * kBookThreads + tid; i < moves; i += step) {
        k.refs[dst[i]] = k.refs[src[i]];
        k.refs[src[i]] = 0;
    }
    const long long total = (long long)k.seqs * k.max_pages;
    for (long long e = rank * kBookThreads + tid; e < total; e += step) {
        const int p = k.table[e];
        if (p < live) continue;
        int lo = 0, hi = moves;            // the first i with src[i] >= p
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (src[mid] < p) lo = mid + 1;
            else hi = mid;
        }
        if (lo < moves && src[lo] == p)
            k.table[e] = dst[lo];
        else
            flag(status, HAD_ERR_INVALID_ARG);
    }
}

// Copies pages within a pool, src[i] -> dst[i]; a pair with a negative index
// is skipped.  HBM-bound: kCopyParts CTAs share a page, each thread moves up to
// four 16-byte words of it at once.  A CTA column y takes the pairs y, y + 512, ...;
// a warp looks at 32 of them with one load each, since most of a list may be
// empty (1501 pages of 43 KB, again and again, so that
// L2 holds part of them: 18 us; 22 us with four words of any array at once and
// the place of each worked out; 19.7 us at 6.6 TB/s).
constexpr int kCopyParts = 4;

// 16-byte words of a page in the three arrays.
struct CopyWords {
    long long codes, kbits, scale;
};

__global__ void __launch_bounds__(256)
cache_copy_kernel(CacheView c, CopyWords words, const int32_t *__restrict__ src,
                  const int32_t *__restrict__ dst, int n, int32_t *status)
{
    const int lane = threadIdx.x & 31;
    for (long long i0 = blockIdx.y; i0 < n; i0 += 32LL * gridDim.y) {
        const long long i = i0 + (long long)lane * gridDim.y;
        const int s = i < n ? __ldg(src + i) : -1, d = i < n ? __ldg(dst + i) : -1;
        const bool pair = s >= 0 && d >= 0, good = pair && s < c.pages && d < c.pages;
        if (pair && !good && blockIdx.x == 0 && threadIdx.x < 32) flag(status, HAD_ERR_INVALID_ARG);
        for (unsigned todo = __ballot_sync(kFullMask, good && s != d); todo; todo &= todo - 1) {
            const int from = __shfl_sync(kFullMask, s, __ffs(todo) - 1);
            const int to = __shfl_sync(kFullMask, d, __ffs(todo) - 1);
            // first words of bits and scales in flight beside those of the codes
            constexpr int kStep = 256 * kCopyParts;
            const long long first = blockIdx.x * 256 + threadIdx.x;
            uint4 *const bits = reinterpret_cast<uint4 *>(c.kbits), *const scale = reinterpret_cast<uint4 *>(c.vscale);
            const uint4 *const bits_from = bits + from * words.kbits, *const scale_from = scale + from * words.scale;
            uint4 *const bits_to = bits + to * words.kbits, *const scale_to = scale + to * words.scale;
            const uint4 *const codes_from = reinterpret_cast<const uint4 *>(c.vcodes) + from * words.codes;
            uint4 *const codes_to = reinterpret_cast<uint4 *>(c.vcodes) + to * words.codes;
            uint4 b, z;
            if (first < words.kbits) b = bits_from[first];
            if (first < words.scale) z = scale_from[first];
            for (long long w = first; w < words.codes; w += 2 * kStep) {
                const bool two = w + kStep < words.codes;
                const uint4 x = codes_from[w];
                uint4 y;
                if (two) y = codes_from[w + kStep];
                codes_to[w] = x;
                if (two) codes_to[w + kStep] = y;
            }
            if (first < words.kbits) bits_to[first] = b;
            if (first < words.scale) scale_to[first] = z;
            for (long long w = first + kStep; w < words.kbits; w += kStep) bits_to[w] = bits_from[w];
            for (long long w = first + kStep; w < words.scale; w += kStep) scale_to[w] = scale_from[w];
        }
    }
}

}  // namespace had
