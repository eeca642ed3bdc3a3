// The paged cache as the kernels see it, and the checks its entry points share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace dspark {

// Status word bits of a cache's workspace, besides kStatusIndex and kStatusTimeout.
constexpr unsigned kStatusCapacity = 4u;

constexpr int kMaxRows = 1024;     // rows of one page operation: one thread block's worth
constexpr int kMaxSeqs = 4096;     // sequences of one attention or append call
constexpr int kMaxPages = 1 << 24;
constexpr int kMaxCtas = 160;      // thread blocks of one attention call (one per SM at most), whatever the device

// Workspace: the status word and the page operations' go flag in the first 256 bytes, the
// attention kernel's arrival counters, then one scratch area that the page operations and the
// attention kernel's partial results use in turn (calls on one workspace never overlap).
constexpr size_t kCacheCountersOffset = 256;
constexpr size_t kCacheScratchOffset = 2048;
static_assert(kCacheCountersOffset + kMaxCtas * 2 * 4 <= kCacheScratchOffset, "counters overlap the scratch area");

struct CacheView {
    unsigned char *pool;
    int *table, *length, *refs;
    unsigned *status;    // [0] status bits, [1] 1 if the page operation goes ahead
    unsigned *counters;
    unsigned char *scratch;
    int num_pages, layers, kv_heads, page_size, page_shift, head_dim, max_seqs, max_pages;
};

// Checks a cache and fills the view; `who` names the entry point in the error text.
dspark_status cache_view(const dspark_cache *c, const char *who, CacheView *v);

// Bytes of the two uses of the scratch area (cache.cu, paged_attention.cu).
size_t cache_ops_scratch_bytes(int max_seqs, int max_pages, int num_pages);
size_t attention_scratch_bytes(int head_dim);

}  // namespace dspark
