// Page operations of the paged cache: allocate (extend), fork, compact, free, copy.
//
// A call's bookkeeping is all or nothing, and the lowest-numbered free pages are taken in a fixed order: the
// arguments are checked, the pages each row needs are counted and added up (a scan over the rows), the free pages are
// counted (a scan over refs), and only then table, length and refs change.  One cluster of up to eight thread blocks does
// it: each block looks at its share of refs and keeps what it found in registers, so refs is read once; the blocks exchange
// their counts, and a free page's number among all free ones says which row takes it (a search in the rows' running
// sums).  Counts are changed by integer atomics, whose order does not change the sums.  Tokens are moved by a second kernel
// that reads what the first one decided.
#include "kv_cache.cuh"
#include "tc.cuh"

namespace dspark {

namespace {

constexpr int kBooksThreads = 1024;
constexpr int kShared = 1 << 30;  // flag in a snapshot entry: the page was shared, the row gets its own

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int kBooksBlocks = 8;  // of one cluster, at most

// Scratch area of the page operations: the rows' own new pages' count (compact), then the snapshot of the rows' old tables.
__device__ __forceinline__ int *scratch_need(const CacheView &c) { return reinterpret_cast<int *>(c.scratch); }
__device__ __forceinline__ int *scratch_snapshot(const CacheView &c) { return scratch_need(c) + kMaxRows; }
size_t snapshot_entries(int max_seqs, int max_pages) { return size_t(max_seqs < kMaxRows ? max_seqs : kMaxRows) * max_pages; }

__device__ __forceinline__ int cluster_block() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return static_cast<int>(r);
}
__device__ __forceinline__ int cluster_blocks() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return static_cast<int>(r);
}
// Every thread of the cluster; orders their memory accesses.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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

// The free pages among refs, kept by the threads that found them: thread t of block b holds the 4 pages from
// (b * rounds + i) * 4096 + 4 t on for each round i of its block, the first 16 rounds in a register, those of larger pools
// in the scratch area (refs may have changed by the time they are wanted).  With few pages to a thread a block's stores to
// the tables fall on few lines (16 pages to a thread took four times as long for 16,000 new pages).
constexpr int kPer = 4, kHeld = 16;

__device__ __forceinline__ unsigned char *scratch_bits(const CacheView &c) {
    return reinterpret_cast<unsigned char *>(scratch_snapshot(c) + size_t(c.max_seqs < kMaxRows ? c.max_seqs : kMaxRows) * c.max_pages);
}

struct FreePages {
    unsigned long long held;  // bits of free pages, four a round
    int rounds, before, count;  // rounds of a block; free pages of earlier blocks, of all (set by find_free)
};

__device__ __forceinline__ unsigned free_bits(const CacheView &c, long long first) {
    if (first + kPer <= c.num_pages) {
        const int4 v = *reinterpret_cast<const int4 *>(c.refs + first);
        return unsigned(v.x == 0) | unsigned(v.y == 0) << 1 | unsigned(v.z == 0) << 2 | unsigned(v.w == 0) << 3;
    }
    unsigned bits = 0;
    for (int q = 0; q < kPer && first + q < c.num_pages; ++q) bits |= unsigned(c.refs[first + q] == 0) << q;
    return bits;
}

__device__ __forceinline__ long long free_first(const FreePages &f, int round) {
    return (static_cast<long long>(cluster_block()) * f.rounds + round) * (kBooksThreads * kPer) + threadIdx.x * kPer;
}

// Counts the free pages of the cluster's blocks; block counts are exchanged through `counts` in every block's shared memory.
// Ends with a cluster barrier: refs may be changed after it.
__device__ void find_free(const CacheView &c, FreePages *f, int *counts, int *warp_sums) {
    const int round = cluster_blocks() * kBooksThreads * kPer;
    f->rounds = (c.num_pages + round - 1) / round;
    f->held = 0;
    const int held = min(f->rounds, kHeld);
#pragma unroll 4
    for (int i = 0; i < held; ++i) f->held |= static_cast<unsigned long long>(free_bits(c, free_first(*f, i))) << (kPer * i);
    int mine = __popcll(f->held);
#pragma unroll 4
    for (int i = kHeld; i < f->rounds; ++i) {
        const unsigned bits = free_bits(c, free_first(*f, i));
        scratch_bits(c)[free_first(*f, i) / kPer] = static_cast<unsigned char>(bits);
        mine += __popc(bits);
    }
    int total = 0;
    block_scan(mine, &total, warp_sums);
    if (threadIdx.x < cluster_blocks()) {
        uint32_t at = smem_addr(counts + cluster_block()), there;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(threadIdx.x));
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there), "r"(total) : "memory");
    }
    cluster_barrier();
    f->before = f->count = 0;
    for (int b = 0; b < cluster_blocks(); ++b) {
        if (b < cluster_block()) f->before += counts[b];
        f->count += counts[b];
    }
}

// Calls give(number, page) for the free pages below `want`, numbered from the lowest.
template <typename Give>
__device__ void give_free(const CacheView &c, const FreePages &f, int want, int *warp_sums, Give give) {
    int at = f.before;
    for (int i = 0; i < f.rounds && at < want; ++i) {  // the same number of turns for the whole block
        unsigned bits = i < kHeld ? static_cast<unsigned>(f.held >> (kPer * i)) & ((1u << kPer) - 1) : scratch_bits(c)[free_first(f, i) / kPer];
        int total = 0, n = at + block_scan(__popc(bits), &total, warp_sums);
        const int first = static_cast<int>(free_first(f, i));
        while (bits && n < want) {
            give(n++, first + __ffs(bits) - 1);
            bits &= bits - 1;
        }
        at += total;
    }
}

// The row whose running sum of needs holds number k: the last r of n with at[r] <= k.
__device__ __forceinline__ int row_of(const int *at, int n, int k) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= k) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Whether the call goes ahead; the first block records why not.  Every block comes to the same answer.
__device__ bool decide(const CacheView &c, bool bad_index, bool full) {
    const int bits = (bad_index ? kStatusIndex : 0) | (full ? kStatusCapacity : 0);
    const bool go = !__syncthreads_or(bits);
    if (cluster_block() == 0) {
        if (bits) atomicOr(c.status, static_cast<unsigned>(bits));
        if (threadIdx.x == 0) c.status[1] = go ? 1u : 0u;
    }
    return go;
}

__global__ void __launch_bounds__(kBooksThreads, 1)
    extend_kernel(CacheView c, const int *rows, const int *counts, int n) {
    __shared__ int warp_sums[32], block_counts[kBooksBlocks];
    __shared__ int s_row[kMaxRows], s_first[kMaxRows], s_at[kMaxRows];
    pdl_launch_dependents();
    cluster_barrier();  // every block has started: its shared memory can be written to
    pdl_wait();
    const int i = threadIdx.x;
    FreePages free;
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
    // rows are at most max_pages each and n at most 1024, but the sum may pass 32 bits: then some prefix does not fit the pool either
    const bool huge = __syncthreads_or(at < 0 || at > c.num_pages || total < 0);
    if (i < n) s_row[i] = row, s_first[i] = pages_of(c, old), s_at[i] = at;
    find_free(c, &free, block_counts, warp_sums);
    if (!decide(c, bad, full || huge || total > free.count)) return;
    if (i < n && cluster_block() == 0) c.length[row] = grown;
    give_free(c, free, total, warp_sums, [&](int k, int page) {
        const int r = row_of(s_at, n, k);
        c.table[size_t(s_row[r]) * c.max_pages + s_first[r] + k - s_at[r]] = page;
        c.refs[page] = 1;
    });
}

__global__ void __launch_bounds__(256) free_kernel(CacheView c, const int *rows, int n) {
    pdl_launch_dependents();
    pdl_wait();
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

__global__ void __launch_bounds__(kBooksThreads, 1)
    fork_books_kernel(CacheView c, const int *src, const int *dst, int n) {
    __shared__ int warp_sums[32], block_counts[kBooksBlocks];
    __shared__ int s_src[kMaxRows], s_dst[kMaxRows], s_at[kMaxRows];
    __shared__ int s_len[kMaxRows], s_old[kMaxRows];  // tokens of the source, and of the target before
    pdl_launch_dependents();
    cluster_barrier();
    pdl_wait();
    const int i = threadIdx.x;
    FreePages free;
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
    find_free(c, &free, block_counts, warp_sums);  // the lengths have been read by every block
    if (!decide(c, bad, total > free.count)) return;
    int *snap = scratch_snapshot(c);
    const int lane = i & 31, first = cluster_block() * (kBooksThreads / 32) + (i >> 5), step = cluster_blocks() * (kBooksThreads / 32);
    for (int r = first; r < n; r += step) {
        if (s_src[r] == s_dst[r]) continue;
        const int *ts = c.table + size_t(s_src[r]) * c.max_pages, *td = c.table + size_t(s_dst[r]) * c.max_pages;
        const int pages = pages_of(c, s_len[r]), old_pages = pages_of(c, s_old[r]);
#pragma unroll 4
        for (int j = lane; j < pages; j += 32) snap[size_t(r) * c.max_pages + j] = ts[j];
#pragma unroll 4
        for (int j = lane; j < old_pages; j += 32) {
            const int page = td[j];
            if (page_ok(c, page)) atomicSub(c.refs + page, 1);
        }
    }
    cluster_barrier();  // every source has been read
    for (int r = first; r < n; r += step) {
        if (s_src[r] == s_dst[r]) continue;
        int *td = c.table + size_t(s_dst[r]) * c.max_pages;
        const int pages = pages_of(c, s_len[r]), whole = s_len[r] >> c.page_shift;
#pragma unroll 4
        for (int j = lane; j < whole; j += 32) {
            const int page = snap[size_t(r) * c.max_pages + j];
            td[j] = page;
            if (page_ok(c, page)) atomicAdd(c.refs + page, 1);
        }
        for (int j = pages + lane; j < pages_of(c, s_old[r]); j += 32) td[j] = -1;
        if (lane == 0) c.length[s_dst[r]] = s_len[r];
    }
    // a row that takes a page has number at[r]; rows that take none share the next one's, and come before it
    give_free(c, free, total, warp_sums, [&](int k, int page) {
        const int r = row_of(s_at, n, k);
        c.table[size_t(s_dst[r]) * c.max_pages + (s_len[r] >> c.page_shift)] = page;
        c.refs[page] = 1;
    });
}

// The filled slots of each forked row's last page: blockIdx.x = `rows` forks next to each other, blockIdx.y = slice of the
// page's layers * 2 * kv_heads runs of head_dim * page_size elements.
//
// Samples of one prompt, next to each other in the list, have one source: a thread keeps the vectors that it has read
// and writes them to each of these forks' pages. 256 samples of 8 prompts, 36 layers (283 MB written, 9 MB of sources; a fill
// of that size takes 40 us): the whole fork 79 us with one fork a block that looks its pages up by itself, 67 with the
// lookups by as many threads at once, 63 with up to four forks a block (eight: 63). 256 forks of 256 prompts, 569 MB: 108,
// 102, 107 us.
constexpr int kForkThreads = 256, kForkVecs = 8, kForkRows = 4;

__global__ void __launch_bounds__(kForkThreads)
    fork_copy_kernel(CacheView c, const int *src, const int *dst, int n, int rows) {
    __shared__ int s_from[kForkRows], s_to[kForkRows], s_slots[kForkRows];
    pdl_launch_dependents();
    pdl_wait();
    if (c.status[1] == 0) return;
    if (threadIdx.x < rows) {
        const int i = blockIdx.x * rows + threadIdx.x;
        int slots = 0;
        if (i < n && src[i] != dst[i]) {
            const int len = c.length[dst[i]], j = len >> c.page_shift;
            slots = len & (c.page_size - 1);
            if (slots != 0) {
                const int from = scratch_snapshot(c)[size_t(i) * c.max_pages + j];
                s_from[threadIdx.x] = from;
                s_to[threadIdx.x] = c.table[size_t(dst[i]) * c.max_pages + j];
                if (!page_ok(c, from)) {
                    if (blockIdx.y == 0) atomicOr(c.status, kStatusIndex);
                    slots = 0;
                }
            }
        }
        s_slots[threadIdx.x] = slots;
    }
    __syncthreads();
    const int runs = c.layers * 2 * c.kv_heads, run_v = c.page_size * c.head_dim / 8;
    const int run0 = static_cast<int>(static_cast<long long>(runs) * blockIdx.y / gridDim.y);
    const int run1 = static_cast<int>(static_cast<long long>(runs) * (blockIdx.y + 1) / gridDim.y);
    uint4 *pool = reinterpret_cast<uint4 *>(c.pool);
    // forks g .. end-1 have one source; its part of this block's runs is one sequence of vectors, eight in flight per thread
    for (int g = 0, end; g < rows; g = end) {
        const int from = s_from[g], slots = s_slots[g];
        for (end = g + 1; end < rows && s_slots[end] == slots && (slots == 0 || s_from[end] == from);) ++end;
        if (slots == 0) continue;
        const int used_v = slots * c.head_dim / 8, count = (run1 - run0) * used_v;
        const uint4 *a = pool + size_t(from) * runs * run_v;
        for (int v0 = threadIdx.x; v0 < count; v0 += kForkThreads * kForkVecs) {
            uint4 x[kForkVecs];
            int at[kForkVecs];
#pragma unroll
            for (int q = 0; q < kForkVecs; ++q) {
                const int v = v0 + q * kForkThreads, run = v / used_v;
                at[q] = (run0 + run) * run_v + v - run * used_v;
                if (v < count) x[q] = ldg_nc_v4(a + at[q]);
            }
            for (int f = g; f < end; ++f) {
                uint4 *b = pool + size_t(s_to[f]) * runs * run_v;
#pragma unroll
                for (int q = 0; q < kForkVecs; ++q)
                    if (v0 + q * kForkThreads < count) __stcs(b + at[q], x[q]);
            }
        }
    }
}

__global__ void __launch_bounds__(kBooksThreads, 1)
    compact_books_kernel(CacheView c, const int *rows, const int *start, const int *kept, int kept_stride, const int *n_kept, int n) {
    __shared__ int warp_sums[32], block_counts[kBooksBlocks];
    __shared__ int s_row[kMaxRows], s_start[kMaxRows], s_len[kMaxRows], s_new[kMaxRows], s_at[kMaxRows];
    __shared__ int s_bad;
    const int i = threadIdx.x, lane = i & 31;
    if (i == 0) s_bad = 0;
    pdl_launch_dependents();
    cluster_barrier();
    pdl_wait();
    FreePages free;
    bool bad = false;
    if (i < n) {
        const int row = rows[i], st = start[i], k = n_kept ? n_kept[i] : 0;
        bad = !row_ok(c, row) || st < 0 || k < 0 || k > kept_stride;
        const int len = bad ? 0 : c.length[row];
        bad |= !length_ok(c, len) || st > len || k > len - st;
        s_row[i] = bad ? 0 : row;
        s_start[i] = bad ? 0 : st;
        s_len[i] = bad ? 0 : len;
        s_new[i] = bad ? 0 : st + k;
    }
    __syncthreads();
    int *snap = scratch_snapshot(c), *needs = scratch_need(c);
    // `per` warps of the cluster to a row, each with a stretch of its list and of its pages
    const int warps = cluster_blocks() * (kBooksThreads / 32);
    const int warp = cluster_block() * (kBooksThreads / 32) + (i >> 5), per = max(1, warps / n), step = warps / per;
    const int part = warp % per;
    for (int r = warp / per; r < n && warp < step * per; r += step) {
        const int st = s_start[r], k = s_new[r] - st, len = s_len[r], pages = pages_of(c, len);
        const int *w = kept + size_t(r) * kept_stride;
        const int k1 = static_cast<int>(static_cast<long long>(k) * (part + 1) / per);
#pragma unroll 4
        for (int j = static_cast<int>(static_cast<long long>(k) * part / per) + lane; j < k1; j += 32) {
            const int at = w[j];
            bad |= at < (j ? w[j - 1] + 1 : st) || at >= len;
        }
        const int *t = c.table + size_t(s_row[r]) * c.max_pages;
        const int lo = st >> c.page_shift, hi = pages_of(c, s_new[r]);
        const int p1 = static_cast<int>(static_cast<long long>(pages) * (part + 1) / per);
        int need = 0;
#pragma unroll 4
        for (int j = static_cast<int>(static_cast<long long>(pages) * part / per) + lane; j < p1; j += 32) {
            const int page = t[j];
            const bool own = j >= lo && j < hi && page_ok(c, page) && c.refs[page] > 1;
            bad |= !page_ok(c, page);
            snap[size_t(r) * c.max_pages + j] = own ? page | kShared : page;
            need += own;
        }
        need = __reduce_add_sync(0xffffffffu, need);
        if (lane == 0) needs[r * per + part] = need;
    }
    // what one block found wrong, every block has to know
    if (bad) {
        for (int b = 0; b < cluster_blocks(); ++b) {
            uint32_t there;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem_addr(&s_bad)), "r"(b));
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there), "r"(1) : "memory");
        }
    }
    find_free(c, &free, block_counts, warp_sums);  // its barrier also orders the needs and the flag
    int total = 0;
    int need = 0;
    if (i < n)
        for (int q = 0; q < per; ++q) need += __ldcg(needs + i * per + q);
    const int at = block_scan(need, &total, warp_sums);
    if (i < n) s_at[i] = at;
    if (!decide(c, s_bad != 0, total > free.count)) return;
    for (int r = warp / per; r < n && warp < step * per; r += step) {
        int *t = c.table + size_t(s_row[r]) * c.max_pages;
        const int last = pages_of(c, s_new[r]), pages = pages_of(c, s_len[r]);
        const int p1 = static_cast<int>(static_cast<long long>(pages) * (part + 1) / per);
#pragma unroll 4
        for (int j = static_cast<int>(static_cast<long long>(pages) * part / per) + lane; j < p1; j += 32) {
            const int entry = snap[size_t(r) * c.max_pages + j];
            if (entry & kShared) {
                atomicSub(c.refs + (entry & ~kShared), 1);
            } else if (j >= last) {
                t[j] = -1;
                atomicSub(c.refs + entry, 1);
            }
        }
        if (lane == 0 && part == 0) c.length[s_row[r]] = s_new[r];
    }
    // the k-th new page of all is the row's (k - at)-th shared one's replacement
    give_free(c, free, total, warp_sums, [&](int k, int page) {
        const int r = row_of(s_at, n, k);
        const int *old = snap + size_t(r) * c.max_pages;
        int j = s_start[r] >> c.page_shift;
        for (int left = k - s_at[r];; ++j)
            if ((old[j] & kShared) && left-- == 0) break;
        c.table[size_t(s_row[r]) * c.max_pages + j] = page;
        c.refs[page] = 1;
    });
}

// Moves the kept tokens of one row (blockIdx.y) in one (layer, k or v, head) run (blockIdx.x) to the front; one warp.
//
// In place and in parallel: token j's new slot is never behind its old one, and both ascend, so a write to slot j only
// lands on the old slot of a token of the same or an earlier tile.  A tile is read whole into shared memory, by
// bulk copies of as many neighbouring tokens as lie together, before it is written; the next tiles' reads are under way
// meanwhile and need no wait for these writes.
//
// A tile is U times 32 tokens, a lane to a token. A step from tile to tile is a chain of a wait and two trips to memory whatever
// the tile's size, so few runs take long tiles (a row of 4000 tokens, 64 runs: the whole compaction 65 us, 74 with tiles of
// 32); of many runs, which memory bounds, short tiles leave room for more blocks on an SM (16 rows of 900-4100 tokens, 64
// runs each: 230 us, 1.3 GB, 247 with tiles of 128).
constexpr int kMoveTokens = 32, kMoveLong = 4, kMoveStages = 4, kMoveAhead = 2;  // two stages on their way, two being written

__device__ __forceinline__ void bulk_load(uint32_t to, const void *from, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from), "r"(bytes),
                 "r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void bulk_store(void *to, uint32_t from, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(from), "r"(bytes) : "memory");
}

// Length, in lanes, of the stretch that begins at this lane if it is a head; `heads` and `active` are ballots.
__device__ __forceinline__ int stretch(unsigned heads, unsigned active, int lane) {
    const unsigned ends = (heads | ~active) & ~((2u << lane) - 1);
    return (ends ? __ffs(ends) - 1 : 32) - lane;
}

template <int U>
__global__ void __launch_bounds__(32) compact_move_kernel(CacheView c, const int *rows, const int *start, const int *kept, int kept_stride,
                                                          const int *n_kept) {
    constexpr int kTokens = U * kMoveTokens;
    extern __shared__ __align__(128) unsigned char stages[];
    __shared__ uint64_t full[kMoveStages];
    __shared__ unsigned char *s_to[kMoveStages][kTokens];
    const int lane = threadIdx.x;
    if (lane == 0) {
        for (int q = 0; q < kMoveStages; ++q) mbar_init(&full[q], 1);
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    __syncwarp();
    pdl_launch_dependents();
    pdl_wait();
    if (c.status[1] == 0) return;
    const int i = blockIdx.y, run = blockIdx.x;
    const int st = start[i], end = st + (n_kept ? n_kept[i] : 0), mask = c.page_size - 1;
    const int *t = c.table + size_t(rows[i]) * c.max_pages;
    const int *snap = scratch_snapshot(c) + size_t(i) * c.max_pages;
    const int *w = kept + size_t(i) * kept_stride;
    const uint32_t token_b = c.head_dim * 2;
    const size_t run_b = size_t(c.page_size) * token_b, page_b = run_b * c.layers * 2 * c.kv_heads;
    unsigned char *pool = c.pool + run * run_b;
    const uint32_t base = smem_addr(stages), stage_b = kTokens * token_b;
    const int first = st & ~mask, tiles = (end - first + kTokens - 1) / kTokens;
    // Looked up ahead, as each is a trip to memory: where two tiles' tokens are now, the pages of one.
    int at[U], next_at[U], from_page[U], to_page[U];
    auto position = [&](int j) { return j >= end || j < st ? j : w[j - st]; };
    auto pages = [&](int u, int j) {
        if (j < end) {
            from_page[u] = snap[at[u] >> c.page_shift];
            to_page[u] = t[j >> c.page_shift];
        }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int j = first + u * kMoveTokens + lane;
        from_page[u] = to_page[u] = 0;
        at[u] = position(j);
        next_at[u] = position(j + kTokens);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) pages(u, first + u * kMoveTokens + lane);
    // stretches of neighbouring tokens that move: whether one begins at the lane, and its length
    auto stretch_at = [&](bool moves, const unsigned char *p, int *length) {
        const unsigned active = __ballot_sync(0xffffffffu, moves);
        const unsigned long long before = __shfl_up_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), 1);
        const bool head = moves && (lane == 0 || !((active >> (lane - 1)) & 1) || before + token_b != reinterpret_cast<unsigned long long>(p));
        *length = stretch(__ballot_sync(0xffffffffu, head), active, lane);
        return head;
    };
    auto load = [&](int tile) {
        const int q = tile % kMoveStages;
        const unsigned char *from[U];
        bool moves[U];
        uint32_t bytes = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = first + tile * kTokens + u * kMoveTokens + lane;
            from[u] = pool + (from_page[u] & ~kShared) * page_b + size_t(at[u] & mask) * token_b;
            unsigned char *to = pool + to_page[u] * page_b + size_t(j & mask) * token_b;
            moves[u] = j < end && from[u] != to;  // the others stay where they are
            s_to[q][u * kMoveTokens + lane] = moves[u] ? to : nullptr;
            bytes += __popc(__ballot_sync(0xffffffffu, moves[u])) * token_b;
            at[u] = next_at[u];
            next_at[u] = position(j + 2 * kTokens);
            pages(u, j + kTokens);
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[q], bytes);
        __syncwarp();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int length;
            if (stretch_at(moves[u], from[u], &length))
                bulk_load(base + q * stage_b + (u * kMoveTokens + lane) * token_b, from[u], length * token_b, &full[q]);
        }
    };
    for (int tile = 0; tile < kMoveAhead && tile < tiles; ++tile) load(tile);
    int loaded = min(tiles, kMoveAhead);
    for (int tile = 0; tile < tiles; ++tile) {
        const int q = tile % kMoveStages;
        if (!__all_sync(0xffffffffu, mbar_wait(&full[q], (tile / kMoveStages) & 1, kDefaultTimeoutNs))) {
            if (lane == 0) atomicOr(c.status, kStatusTimeout);
            break;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            unsigned char *to = s_to[q][u * kMoveTokens + lane];
            int length;
            if (stretch_at(to != nullptr, to, &length))
                bulk_store(to, base + q * stage_b + (u * kMoveTokens + lane) * token_b, length * token_b);
        }
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        if (tile + kMoveAhead < tiles) {
            // the slot's last tile has been written from it
            asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kMoveStages - kMoveAhead) : "memory");
            __syncwarp();
            load(tile + kMoveAhead);
            ++loaded;
        }
    }
    // copies in flight end before the block does, also after a wait that gave up
    for (int tile = max(loaded - kMoveStages, 0); tile < loaded; ++tile)
        mbar_wait(&full[tile % kMoveStages], (tile / kMoveStages) & 1, kDefaultTimeoutNs);
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__global__ void __launch_bounds__(256) copy_pages_kernel(CacheView c, const int *src, const int *dst, size_t page_v) {
    pdl_launch_dependents();
    pdl_wait();
    const int i = blockIdx.x, a = src[i], b = dst[i];
    if (!page_ok(c, a) || !page_ok(c, b)) {
        if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(c.status, kStatusIndex);
        return;
    }
    const uint4 *from = reinterpret_cast<const uint4 *>(c.pool) + a * page_v;
    uint4 *to = reinterpret_cast<uint4 *>(c.pool) + b * page_v;
    const size_t step = size_t(gridDim.y) * blockDim.x;
    for (size_t v0 = size_t(blockIdx.y) * blockDim.x + threadIdx.x; v0 < page_v; v0 += 4 * step) {
        uint4 x[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (v0 + q * step < page_v) x[q] = ldg_nc_v4(from + v0 + q * step);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (v0 + q * step < page_v) to[v0 + q * step] = x[q];
    }
}

dspark_status launched(cudaError_t e, const char *what) { return e == cudaSuccess ? DSPARK_OK : cuda_fail(e, what); }

// Launches the books of a call that looks through `entries` of lists and tables: a block for each 4096 of them or of the pool's pages, up
// to eight (1, 2, 4 or 8).  Compacting 16 rows of 2,500 tokens took 233 us with eight, 245 with one.
template <typename... KArgs, typename... Args>
cudaError_t launch_books(void (*kernel)(KArgs...), const CacheView &c, long long entries, cudaStream_t stream, Args &&...args) {
    const long long work = entries > c.num_pages ? entries : c.num_pages;
    unsigned blocks = 1;
    while (blocks < kBooksBlocks && static_cast<long long>(blocks) * kBooksThreads * kPer < work) blocks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kBooksThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...);
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

size_t cache_ops_scratch_bytes(int max_seqs, int max_pages, int num_pages) {
    const size_t bits = (size_t(num_pages) / (kBooksThreads * kPer) + kBooksBlocks) * kBooksThreads;  // a byte for four pages
    return up256(4 * (kMaxRows + snapshot_entries(max_seqs, max_pages)) + bits);
}

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
    const size_t ops = cache_ops_scratch_bytes(c->max_seqs, c->max_pages, c->num_pages), att = attention_scratch_bytes(c->head_dim);
    return kCacheScratchOffset + (ops > att ? ops : att);
}

extern "C" dspark_status dspark_cache_extend(const dspark_cache *cache, const int32_t *rows, const int32_t *counts, int n,
                                             dspark_stream_t stream) {
    CacheView c;
    dspark_status st = cache_view(cache, "cache_extend", &c);
    if (st != DSPARK_OK || (st = check_rows("cache_extend", c, rows, counts, n)) != DSPARK_OK || n == 0) return st;
    return launched(launch_books(extend_kernel, c, static_cast<long long>(n) * 128, stream, c, rows, counts, n), "cache_extend");
}

extern "C" dspark_status dspark_cache_free(const dspark_cache *cache, const int32_t *rows, int n, dspark_stream_t stream) {
    CacheView c;
    dspark_status st = cache_view(cache, "cache_free", &c);
    if (st != DSPARK_OK || (st = check_rows("cache_free", c, rows, rows, n)) != DSPARK_OK || n == 0) return st;
    return launched(launch_pdl(free_kernel, dim3(n), dim3(256), 0, stream, c, rows, n), "cache_free");
}

extern "C" dspark_status dspark_cache_fork(const dspark_cache *cache, const int32_t *src, const int32_t *dst, int n,
                                           dspark_stream_t stream) {
    CacheView c;
    dspark_status st = cache_view(cache, "cache_fork", &c);
    if (st != DSPARK_OK || (st = check_rows("cache_fork", c, src, dst, n)) != DSPARK_OK || n == 0) return st;
    st = launched(launch_books(fork_books_kernel, c, static_cast<long long>(n) * c.max_pages, stream, c, src, dst, n), "cache_fork");
    if (st != DSPARK_OK) return st;
    int sms = 0;
    if ((st = static_cast<dspark_status>(current_sm_count(&sms))) != DSPARK_OK) return st;
    // Slices of a page: as many as give each thread its eight vectors of a full one. Forks of a block: as many as leave four
    // rounds of the SMs of such slices; then no more blocks than those four rounds, as each begins with a chain of lookups.
    const long long full = 2ll * c.layers * c.kv_heads * c.page_size * c.head_dim / 8 / (kForkThreads * kForkVecs);
    const long long four = 4ll * 6 * sms, share = full * n / four;
    const int rows_of = share < 1 ? 1 : share < kForkRows ? static_cast<int>(share) : kForkRows, blocks = (n + rows_of - 1) / rows_of;
    const long long most = four / blocks;
    const unsigned slices = static_cast<unsigned>(full < 1 || most < 1 ? 1 : full < most ? full : most);
    return launched(launch_pdl(fork_copy_kernel, dim3(blocks, slices), dim3(kForkThreads), 0, stream, c, src, dst, n, rows_of), "cache_fork");
}

extern "C" dspark_status dspark_cache_compact(const dspark_cache *cache, const int32_t *rows, const int32_t *start,
                                              const int32_t *kept, int kept_stride, const int32_t *n_kept, int n,
                                              dspark_stream_t stream) {
    CacheView c;
    dspark_status st = cache_view(cache, "cache_compact", &c);
    if (st != DSPARK_OK || (st = check_rows("cache_compact", c, rows, start, n)) != DSPARK_OK) return st;
    if (kept_stride < 0) return fail(DSPARK_ERR_INVALID, "cache_compact: kept_stride=%d is negative", kept_stride);
    if (n == 0) return DSPARK_OK;
    if (kept_stride > 0 && (!kept || !n_kept)) return fail(DSPARK_ERR_INVALID, "cache_compact: null pointer argument");
    const long long entries = static_cast<long long>(n) * (kept_stride + c.max_pages);
    st = launched(launch_books(compact_books_kernel, c, entries, stream, c, rows, start, kept, kept_stride, n_kept, n), "cache_compact");
    if (st != DSPARK_OK) return st;
    int sms = 0;
    if ((st = static_cast<dspark_status>(current_sm_count(&sms))) != DSPARK_OK) return st;
    const int runs = c.layers * 2 * c.kv_heads;
    const bool few = static_cast<long long>(runs) * n <= sms;  // an SM to each run
    auto *kernel = few ? compact_move_kernel<kMoveLong> : compact_move_kernel<1>;
    const int tile_b = kMoveStages * kMoveTokens * 2;  // for each unit of head_dim
    if (few) {
        static int configured = -1;
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess && configured != dev) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoveLong * tile_b * 128);
            if (e == cudaSuccess) configured = dev;
        }
        if (e != cudaSuccess) return cuda_fail(e, "cache_compact");
    }
    return launched(launch_pdl(kernel, dim3(runs, n), dim3(32), size_t(few ? kMoveLong : 1) * tile_b * c.head_dim, stream, c, rows, start,
                               kept, kept_stride, n_kept),
                    "cache_compact");
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
    const dim3 grid(n, static_cast<unsigned>(blocks < 64 ? blocks : 64));
    return launched(launch_pdl(copy_pages_kernel, grid, dim3(256), 0, stream, c, src, dst, page_v), "cache_copy_pages");
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
    // A wait that gave up may have ended attention's blocks between their arrivals at a join: their counts start anew as well.
    e = cudaMemsetAsync(c.status, 0, bits & kStatusTimeout ? kCacheScratchOffset : 4, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return cuda_fail(e, "cache_status");
    if (bits & kStatusTimeout) return fail(DSPARK_ERR_TIMEOUT, "paged cache: a device-side wait gave up");
    if (bits & kStatusIndex) return fail(DSPARK_ERR_INDEX, "paged cache: a row, token or page index was out of range");
    return fail(DSPARK_ERR_CAPACITY, "paged cache: not enough free pages, or a row is full");
}
