// Page operations of the paged cache: allocate (extend), fork, compact, free, copy.
//
// A call's bookkeeping is decided by one thread block, so that it is all or nothing and the
// lowest-numbered free pages are taken in a fixed order: it checks the arguments, counts the
// pages each row needs, adds the counts up (a scan over the rows), finds that many free pages
// (a scan over refs) and only then changes table, length and refs.  Counts are changed by integer
// atomics, whose order does not change the sums.  Tokens are moved by a second kernel that reads
// what the first one decided.
#include "kv_cache.cuh"

namespace dspark {

namespace {

constexpr int kBooksThreads = 1024;
constexpr int kShared = 1 << 30;  // flag in a snapshot entry: the page was shared, the row gets its own

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Scratch area of the page operations: fresh pages, then the snapshot of the rows' old tables.
__device__ __forceinline__ int *scratch_fresh(const CacheView &c) { return reinterpret_cast<int *>(c.scratch); }
__host__ __device__ inline size_t fresh_entries(int max_seqs, int max_pages) {
    return size_t(max_seqs < kMaxRows ? max_seqs : kMaxRows) * max_pages;
}
__device__ __forceinline__ int *scratch_snapshot(const CacheView &c) {
    return scratch_fresh(c) + fresh_entries(c.max_seqs, c.max_pages);
}

__device__ __forceinline__ bool page_ok(const CacheView &c, int page) {
    return static_cast<unsigned>(page) < static_cast<unsigned>(c.num_pages);
}
__device__ __forceinline__ bool row_ok(const CacheView &c, int row) {
    return static_cast<unsigned>(row) < static_cast<unsigned>(c.max_seqs);
}
__device__ __forceinline__ int pages_of(const CacheView &c, int tokens) {
    return (tokens + c.page_size - 1) >> c.page_shift;
}
__device__ __forceinline__ bool length_ok(const CacheView &c, int tokens) {
    return tokens >= 0 && tokens <= static_cast<long long>(c.max_pages) * c.page_size;
}

// Exclusive scan over the block's threads in thread order; *total is the sum.
__device__ int block_scan(int v, int *total, int *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // warp_sums may still be read from the last call
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = lane < static_cast<int>(blockDim.x >> 5) ? warp_sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    *total = warp_sums[31];
    return x - v + (warp ? warp_sums[warp - 1] : 0);
}

// The `want` lowest-numbered free pages, ascending, to out[0..want); false if there are fewer.
__device__ bool find_free(const CacheView &c, int want, int *out, int *warp_sums) {
    constexpr int kPer = 16;
    int found = 0;
    for (int base = 0; base < c.num_pages && found < want; base += kBooksThreads * kPer) {
        const int p0 = base + static_cast<int>(threadIdx.x) * kPer;
        unsigned free = 0;
        if (p0 + kPer <= c.num_pages) {
            const int4 *r = reinterpret_cast<const int4 *>(c.refs + p0);
#pragma unroll
            for (int q = 0; q < kPer / 4; ++q) {
                const int4 v = r[q];
                free |= (unsigned(v.x == 0) | unsigned(v.y == 0) << 1 | unsigned(v.z == 0) << 2 | unsigned(v.w == 0) << 3)
                        << (4 * q);
            }
        } else {
            for (int q = 0; q < kPer && p0 + q < c.num_pages; ++q) free |= unsigned(c.refs[p0 + q] == 0) << q;
        }
        int total = 0;
        int at = found + block_scan(__popc(free), &total, warp_sums);
        while (free && at < want) {
            out[at++] = p0 + __ffs(free) - 1;
            free &= free - 1;
        }
        found += total;
    }
    __syncthreads();
    return found >= want;
}

// Whether the call goes ahead; records why not.
__device__ bool decide(const CacheView &c, bool bad_index, bool full) {
    const int bits = (bad_index ? kStatusIndex : 0) | (full ? kStatusCapacity : 0);
    const bool go = !__syncthreads_or(bits);
    if (bits) atomicOr(c.status, static_cast<unsigned>(bits));
    if (threadIdx.x == 0) c.status[1] = go ? 1u : 0u;
    return go;
}

__global__ void __launch_bounds__(kBooksThreads) extend_kernel(CacheView c, const int *rows, const int *counts, int n) {
    __shared__ int warp_sums[32];
    __shared__ int s_row[kMaxRows], s_first[kMaxRows], s_need[kMaxRows], s_at[kMaxRows];
    const int i = threadIdx.x;
    bool bad = false, full = false;
    int row = 0, old = 0, grown = 0, need = 0;
    if (i < n) {
        row = rows[i];
        const int add = counts[i];
        bad = !row_ok(c, row) || add < 0;
        if (!bad) {
            old = c.length[row];
            bad = !length_ok(c, old);
            full = !bad && static_cast<long long>(old) + add > static_cast<long long>(c.max_pages) * c.page_size;
            if (!bad && !full) {
                grown = old + add;
                need = pages_of(c, grown) - pages_of(c, old);
            }
        }
    }
    int total = 0;
    const int at = block_scan(need, &total, warp_sums);
    if (i < n) s_row[i] = row, s_first[i] = pages_of(c, old), s_need[i] = need, s_at[i] = at;
    int *fresh = scratch_fresh(c);
    const bool enough = total <= c.num_pages && find_free(c, total, fresh, warp_sums);
    if (!decide(c, bad, full || !enough)) return;
    if (i < n) c.length[row] = grown;
    for (int r = i >> 5; r < n; r += kBooksThreads / 32) {
        int *t = c.table + size_t(s_row[r]) * c.max_pages + s_first[r];
        for (int j = i & 31; j < s_need[r]; j += 32) {
            const int page = fresh[s_at[r] + j];
            t[j] = page;
            c.refs[page] = 1;
        }
    }
}

__global__ void __launch_bounds__(256) free_kernel(CacheView c, const int *rows, int n) {
    bool bad = false;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int row = rows[i];
        bad |= !row_ok(c, row) || !length_ok(c, c.length[row]);
    }
    // Rows are distinct, so the only length this block may find changed by another is set to 0.
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) atomicOr(c.status, kStatusIndex);
        return;
    }
    const int row = rows[blockIdx.x];
    int *t = c.table + size_t(row) * c.max_pages;
    const int pages = pages_of(c, c.length[row]);
    __syncthreads();
    if (threadIdx.x == 0) c.length[row] = 0;
    for (int j = threadIdx.x; j < pages; j += blockDim.x) {
        const int page = t[j];
        if (page_ok(c, page)) atomicSub(c.refs + page, 1);
        t[j] = -1;
    }
}

__global__ void __launch_bounds__(kBooksThreads) fork_books_kernel(CacheView c, const int *src, const int *dst, int n) {
    __shared__ int warp_sums[32];
    __shared__ int s_src[kMaxRows], s_dst[kMaxRows], s_at[kMaxRows];
    __shared__ int s_len[kMaxRows], s_old[kMaxRows];  // tokens of the source, and of the target before
    const int i = threadIdx.x;
    bool bad = false;
    int s = 0, d = 0, len = 0, old = 0;
    if (i < n) {
        s = src[i];
        d = dst[i];
        bad = !row_ok(c, s) || !row_ok(c, d);
        if (!bad) {
            len = c.length[s];
            old = c.length[d];
            bad = !length_ok(c, len) || !length_ok(c, old);
        }
    }
    const int need = i < n && !bad && s != d && (len & (c.page_size - 1)) ? 1 : 0;
    int total = 0;
    const int at = block_scan(need, &total, warp_sums);
    if (i < n) s_src[i] = s, s_dst[i] = d, s_len[i] = len, s_old[i] = old, s_at[i] = at;
    int *fresh = scratch_fresh(c), *snap = scratch_snapshot(c);
    const bool enough = total <= c.num_pages && find_free(c, total, fresh, warp_sums);
    if (!decide(c, bad, !enough)) return;
    const int lane = i & 31;
    for (int r = i >> 5; r < n; r += kBooksThreads / 32) {
        if (s_src[r] == s_dst[r]) continue;
        const int *ts = c.table + size_t(s_src[r]) * c.max_pages, *td = c.table + size_t(s_dst[r]) * c.max_pages;
        for (int j = lane; j < pages_of(c, s_len[r]); j += 32) snap[size_t(r) * c.max_pages + j] = ts[j];
        for (int j = lane; j < pages_of(c, s_old[r]); j += 32) {
            const int page = td[j];
            if (page_ok(c, page)) atomicSub(c.refs + page, 1);
        }
    }
    __syncthreads();
    for (int r = i >> 5; r < n; r += kBooksThreads / 32) {
        if (s_src[r] == s_dst[r]) continue;
        int *td = c.table + size_t(s_dst[r]) * c.max_pages;
        const int pages = pages_of(c, s_len[r]), full = s_len[r] >> c.page_shift;
        for (int j = lane; j < pages; j += 32) {
            const int page = j < full ? snap[size_t(r) * c.max_pages + j] : fresh[s_at[r]];
            td[j] = page;
            if (page_ok(c, page)) atomicAdd(c.refs + page, 1);
        }
        for (int j = pages + lane; j < pages_of(c, s_old[r]); j += 32) td[j] = -1;
        if (lane == 0) c.length[s_dst[r]] = s_len[r];
    }
}

// The filled slots of each forked row's last page: blockIdx.x = fork, blockIdx.y = slice of the page's
// layers * 2 * kv_heads runs of head_dim * page_size elements.
__global__ void __launch_bounds__(256) fork_copy_kernel(CacheView c, const int *src, const int *dst) {
    if (c.status[1] == 0) return;
    const int i = blockIdx.x;
    const int d = dst[i];
    if (src[i] == d) return;
    const int len = c.length[d], slots = len & (c.page_size - 1);
    if (slots == 0) return;
    const int j = len >> c.page_shift;
    const int from = scratch_snapshot(c)[size_t(i) * c.max_pages + j], to = c.table[size_t(d) * c.max_pages + j];
    if (!page_ok(c, from)) {
        if (threadIdx.x == 0) atomicOr(c.status, kStatusIndex);
        return;
    }
    const int runs = c.layers * 2 * c.kv_heads;
    const int run_v = c.page_size * c.head_dim / 8, used_v = slots * c.head_dim / 8;
    const uint4 *a = reinterpret_cast<const uint4 *>(c.pool) + size_t(from) * runs * run_v;
    uint4 *b = reinterpret_cast<uint4 *>(c.pool) + size_t(to) * runs * run_v;
    for (int run = blockIdx.y; run < runs; run += gridDim.y)
        for (int v = threadIdx.x; v < used_v; v += blockDim.x) b[size_t(run) * run_v + v] = a[size_t(run) * run_v + v];
}

__global__ void __launch_bounds__(kBooksThreads) compact_books_kernel(CacheView c, const int *rows, const int *start,
                                                                      const int *kept, int kept_stride,
                                                                      const int *n_kept, int n) {
    __shared__ int warp_sums[32];
    __shared__ int s_row[kMaxRows], s_start[kMaxRows], s_len[kMaxRows], s_new[kMaxRows], s_need[kMaxRows];
    const int i = threadIdx.x, lane = i & 31;
    bool bad = false;
    if (i < n) {
        const int row = rows[i], st = start[i], k = n_kept[i];
        bad = !row_ok(c, row) || st < 0 || k < 0 || k > kept_stride;
        const int len = bad ? 0 : c.length[row];
        bad |= !length_ok(c, len) || st > len || k > len - st;
        s_row[i] = bad ? 0 : row;
        s_start[i] = bad ? 0 : st;
        s_len[i] = bad ? 0 : len;
        s_new[i] = bad ? 0 : st + k;
    }
    __syncthreads();
    int *fresh = scratch_fresh(c), *snap = scratch_snapshot(c);
    for (int r = i >> 5; r < n; r += kBooksThreads / 32) {
        const int st = s_start[r], k = s_new[r] - st, len = s_len[r];
        const int *w = kept + size_t(r) * kept_stride;
        for (int j = lane; j < k; j += 32) {
            const int at = w[j];
            bad |= at < (j ? w[j - 1] + 1 : st) || at >= len;
        }
        const int *t = c.table + size_t(s_row[r]) * c.max_pages;
        const int first = st >> c.page_shift, last = pages_of(c, s_new[r]);
        int need = 0;
        for (int j = lane; j < pages_of(c, len); j += 32) {
            const int page = t[j];
            const bool own = j >= first && j < last && page_ok(c, page) && c.refs[page] > 1;
            bad |= !page_ok(c, page);
            snap[size_t(r) * c.max_pages + j] = own ? page | kShared : page;
            need += own;
        }
        need = __reduce_add_sync(0xffffffffu, need);
        if (lane == 0) s_need[r] = need;
    }
    __syncthreads();
    int total = 0;
    const int at = block_scan(i < n ? s_need[i] : 0, &total, warp_sums);
    __syncthreads();
    if (i < n) s_need[i] = at;
    const bool enough = total <= c.num_pages && find_free(c, total, fresh, warp_sums);
    if (!decide(c, bad, !enough)) return;
    for (int r = i >> 5; r < n; r += kBooksThreads / 32) {
        int *t = c.table + size_t(s_row[r]) * c.max_pages;
        const int last = pages_of(c, s_new[r]), pages = pages_of(c, s_len[r]);
        int next = s_need[r];
        for (int j0 = 0; j0 < pages; j0 += 32) {
            const int j = j0 + lane;
            const int entry = j < pages ? snap[size_t(r) * c.max_pages + j] : 0;
            const bool own = (entry & kShared) != 0, drop = j >= last && j < pages;
            const unsigned mine = __ballot_sync(0xffffffffu, own);
            if (own) {
                const int page = fresh[next + __popc(mine & ((1u << lane) - 1))];
                t[j] = page;
                c.refs[page] = 1;
                atomicSub(c.refs + (entry & ~kShared), 1);
            } else if (drop) {
                t[j] = -1;
                atomicSub(c.refs + entry, 1);
            }
            next += __popc(mine);
        }
        if (lane == 0) c.length[s_row[r]] = s_new[r];
    }
}

// Moves the kept tokens of one row (blockIdx.y) in one (layer, k or v, head) run (blockIdx.x) to the front.
//
// In place and in parallel: token j's new slot is never behind its old one, and both ascend, so a write to
// slot j only lands on the old slot of a token that was read before.  A tile of tokens is therefore read whole
// into registers, and written after a barrier; the next tile's reads need no wait for these writes.
constexpr int kMoveThreads = 256, kMoveVecs = 8;

__global__ void __launch_bounds__(kMoveThreads) compact_move_kernel(CacheView c, const int *rows, const int *start,
                                                                    const int *kept, int kept_stride, const int *n_kept) {
    if (c.status[1] == 0) return;
    const int i = blockIdx.y, run = blockIdx.x;
    const int st = start[i], end = st + n_kept[i];
    const int *t = c.table + size_t(rows[i]) * c.max_pages;
    const int *snap = scratch_snapshot(c) + size_t(i) * c.max_pages;
    const int *w = kept + size_t(i) * kept_stride;
    const int vecs = c.head_dim / 8;                       // 16-byte vectors of a token: 8 or 16
    const int per = kMoveThreads / vecs * kMoveVecs;       // tokens of a tile
    const int vec = threadIdx.x % vecs, sub = threadIdx.x / vecs, step = kMoveThreads / vecs;
    const size_t run_v = size_t(c.page_size) * vecs, page_v = run_v * c.layers * 2 * c.kv_heads;
    uint4 *pool = reinterpret_cast<uint4 *>(c.pool) + run * run_v + vec;
    const int mask = c.page_size - 1;
    for (int j0 = st & ~mask; j0 < end; j0 += per) {
        uint4 x[kMoveVecs];
        size_t to[kMoveVecs];
#pragma unroll
        for (int q = 0; q < kMoveVecs; ++q) {
            const int j = j0 + q * step + sub;
            to[q] = ~size_t(0);
            if (j < end) {
                const int s = j < st ? j : w[j - st];
                const int from = snap[s >> c.page_shift] & ~kShared, page = t[j >> c.page_shift];
                if (from != page || s != j) {
                    to[q] = page * page_v + size_t(j & mask) * vecs;
                    x[q] = pool[from * page_v + size_t(s & mask) * vecs];
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kMoveVecs; ++q)
            if (to[q] != ~size_t(0)) pool[to[q]] = x[q];
    }
}

__global__ void __launch_bounds__(256) copy_pages_kernel(CacheView c, const int *src, const int *dst, size_t page_v) {
    const int i = blockIdx.x, a = src[i], b = dst[i];
    if (!page_ok(c, a) || !page_ok(c, b)) {
        if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(c.status, kStatusIndex);
        return;
    }
    const uint4 *from = reinterpret_cast<const uint4 *>(c.pool) + a * page_v;
    uint4 *to = reinterpret_cast<uint4 *>(c.pool) + b * page_v;
    for (size_t v = size_t(blockIdx.y) * blockDim.x + threadIdx.x; v < page_v; v += size_t(gridDim.y) * blockDim.x)
        to[v] = from[v];
}

dspark_status launched(const char *what) {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DSPARK_OK : cuda_fail(e, what);
}

dspark_status check_rows(const char *who, const CacheView &c, const void *a, const void *b, int n) {
    if (n < 0) return fail(DSPARK_ERR_INVALID, "%s: n=%d is negative", who, n);
    if (n > kMaxRows) return fail(DSPARK_ERR_UNSUPPORTED, "%s: n=%d rows, at most %d in one call", who, n, kMaxRows);
    if (n > c.max_seqs) return fail(DSPARK_ERR_INVALID, "%s: n=%d rows of a table of %d", who, n, c.max_seqs);
    if (n > 0 && (!a || !b)) return fail(DSPARK_ERR_INVALID, "%s: null pointer argument", who);
    return DSPARK_OK;
}

bool sizes_ok(const dspark_cache *c) {
    const int ps = c->page_size;
    return c->num_pages >= 1 && c->num_pages < kMaxPages && c->layers >= 1 && c->kv_heads >= 1 && c->max_seqs >= 1 &&
           c->max_pages >= 1 && ps >= 16 && ps <= 256 && (ps & (ps - 1)) == 0 &&
           (c->head_dim == 64 || c->head_dim == 128) && (c->dtype == DSPARK_FP16 || c->dtype == DSPARK_BF16) &&
           static_cast<long long>(c->max_pages) * ps < (1ll << 30) &&
           2ll * c->layers * c->kv_heads * ps * c->head_dim < (1ll << 31);
}

}  // namespace

size_t cache_ops_scratch_bytes(int max_seqs, int max_pages) { return up256(2 * 4 * fresh_entries(max_seqs, max_pages)); }

dspark_status cache_view(const dspark_cache *c, const char *who, CacheView *v) {
    clear_error();
    if (!c) return fail(DSPARK_ERR_INVALID, "%s: null cache", who);
    if (c->num_pages < 1 || c->layers < 1 || c->kv_heads < 1 || c->max_seqs < 1 || c->max_pages < 1)
        return fail(DSPARK_ERR_INVALID, "%s: bad cache sizes pages=%d layers=%d kv_heads=%d max_seqs=%d max_pages=%d", who,
                    c->num_pages, c->layers, c->kv_heads, c->max_seqs, c->max_pages);
    if (!sizes_ok(c))
        return fail(DSPARK_ERR_UNSUPPORTED,
                    "%s: cache of page_size %d, head_dim %d, dtype %d, %d pages (page_size 16..256, a power of two; "
                    "head_dim 64 or 128; fp16 or bf16; fewer than 2^24 pages, 2^30 tokens of a row and 2^31 elements of a page)",
                    who, c->page_size, c->head_dim, c->dtype, c->num_pages);
    if (!c->pool || !c->table || !c->length || !c->refs || !c->workspace)
        return fail(DSPARK_ERR_INVALID, "%s: null pointer in the cache", who);
    if (!aligned(c->pool, 16) || !aligned(c->refs, 16) || !aligned(c->table, 4) || !aligned(c->length, 4) ||
        !aligned(c->workspace, 256))
        return fail(DSPARK_ERR_INVALID, "%s: pool and refs must be 16-byte and the workspace 256-byte aligned", who);
    const size_t need = dspark_cache_workspace_bytes(c);
    if (c->workspace_bytes < need)
        return fail(DSPARK_ERR_INVALID, "%s: workspace of %zu bytes, %zu needed", who, c->workspace_bytes, need);
    unsigned char *ws = static_cast<unsigned char *>(c->workspace);
    v->pool = static_cast<unsigned char *>(c->pool);
    v->table = c->table;
    v->length = c->length;
    v->refs = c->refs;
    v->status = reinterpret_cast<unsigned *>(ws);
    v->counters = reinterpret_cast<unsigned *>(ws + kCacheCountersOffset);
    v->scratch = ws + kCacheScratchOffset;
    v->num_pages = c->num_pages;
    v->layers = c->layers;
    v->kv_heads = c->kv_heads;
    v->page_size = c->page_size;
    v->page_shift = __builtin_ctz(static_cast<unsigned>(c->page_size));
    v->head_dim = c->head_dim;
    v->max_seqs = c->max_seqs;
    v->max_pages = c->max_pages;
    return DSPARK_OK;
}

}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_cache_workspace_bytes(const dspark_cache *c) {
    if (!c || !sizes_ok(c)) return 0;
    const size_t ops = cache_ops_scratch_bytes(c->max_seqs, c->max_pages), att = attention_scratch_bytes(c->head_dim);
    return kCacheScratchOffset + (ops > att ? ops : att);
}

extern "C" dspark_status dspark_cache_extend(const dspark_cache *cache, const int32_t *rows, const int32_t *counts, int n,
                                             dspark_stream_t stream) {
    CacheView c;
    dspark_status st = cache_view(cache, "cache_extend", &c);
    if (st != DSPARK_OK || (st = check_rows("cache_extend", c, rows, counts, n)) != DSPARK_OK || n == 0) return st;
    extend_kernel<<<1, kBooksThreads, 0, stream>>>(c, rows, counts, n);
    return launched("cache_extend");
}

extern "C" dspark_status dspark_cache_free(const dspark_cache *cache, const int32_t *rows, int n, dspark_stream_t stream) {
    CacheView c;
    dspark_status st = cache_view(cache, "cache_free", &c);
    if (st != DSPARK_OK || (st = check_rows("cache_free", c, rows, rows, n)) != DSPARK_OK || n == 0) return st;
    free_kernel<<<n, 256, 0, stream>>>(c, rows, n);
    return launched("cache_free");
}

extern "C" dspark_status dspark_cache_fork(const dspark_cache *cache, const int32_t *src, const int32_t *dst, int n,
                                           dspark_stream_t stream) {
    CacheView c;
    dspark_status st = cache_view(cache, "cache_fork", &c);
    if (st != DSPARK_OK || (st = check_rows("cache_fork", c, src, dst, n)) != DSPARK_OK || n == 0) return st;
    fork_books_kernel<<<1, kBooksThreads, 0, stream>>>(c, src, dst, n);
    const int runs = c.layers * 2 * c.kv_heads;
    fork_copy_kernel<<<dim3(n, runs < 64 ? runs : 64), 256, 0, stream>>>(c, src, dst);
    return launched("cache_fork");
}

extern "C" dspark_status dspark_cache_compact(const dspark_cache *cache, const int32_t *rows, const int32_t *start,
                                              const int32_t *kept, int kept_stride, const int32_t *n_kept, int n,
                                              dspark_stream_t stream) {
    CacheView c;
    dspark_status st = cache_view(cache, "cache_compact", &c);
    if (st != DSPARK_OK || (st = check_rows("cache_compact", c, rows, start, n)) != DSPARK_OK) return st;
    if (kept_stride < 0) return fail(DSPARK_ERR_INVALID, "cache_compact: kept_stride=%d is negative", kept_stride);
    if (n == 0) return DSPARK_OK;
    if (!n_kept || (!kept && kept_stride > 0)) return fail(DSPARK_ERR_INVALID, "cache_compact: null pointer argument");
    compact_books_kernel<<<1, kBooksThreads, 0, stream>>>(c, rows, start, kept, kept_stride, n_kept, n);
    compact_move_kernel<<<dim3(c.layers * 2 * c.kv_heads, n), kMoveThreads, 0, stream>>>(c, rows, start, kept, kept_stride,
                                                                                         n_kept);
    return launched("cache_compact");
}

extern "C" dspark_status dspark_cache_copy_pages(const dspark_cache *cache, const int32_t *src, const int32_t *dst, int n,
                                                 dspark_stream_t stream) {
    CacheView c;
    dspark_status st = cache_view(cache, "cache_copy_pages", &c);
    if (st != DSPARK_OK) return st;
    if (n < 0) return fail(DSPARK_ERR_INVALID, "cache_copy_pages: n=%d is negative", n);
    if (n == 0) return DSPARK_OK;
    if (!src || !dst) return fail(DSPARK_ERR_INVALID, "cache_copy_pages: null pointer argument");
    const size_t page_v = size_t(c.layers) * 2 * c.kv_heads * c.page_size * c.head_dim / 8;
    const size_t blocks = (page_v + 1023) / 1024;
    copy_pages_kernel<<<dim3(n, static_cast<unsigned>(blocks < 64 ? blocks : 64)), 256, 0, stream>>>(c, src, dst, page_v);
    return launched("cache_copy_pages");
}

extern "C" dspark_status dspark_cache_status(const dspark_cache *cache, dspark_stream_t stream) {
    CacheView c;
    dspark_status st = cache_view(cache, "cache_status", &c);
    if (st != DSPARK_OK) return st;
    unsigned bits = 0;
    cudaError_t e = cudaMemcpyAsync(&bits, c.status, 4, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return cuda_fail(e, "cache_status");
    if (bits == 0) return DSPARK_OK;
    e = cudaMemsetAsync(c.status, 0, 4, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return cuda_fail(e, "cache_status");
    if (bits & kStatusTimeout) return fail(DSPARK_ERR_TIMEOUT, "paged cache: a device-side wait gave up");
    if (bits & kStatusIndex) return fail(DSPARK_ERR_INDEX, "paged cache: a row, token or page index was out of range");
    return fail(DSPARK_ERR_CAPACITY, "paged cache: not enough free pages, or a row is full");
}
