// Attention of a chunk of new tokens over the paged cache.
//
// One warp to a (token, query head): the lanes share the head's elements, and the keys that the token
// sees are taken one after another with the running maximum and sum of the softmax.
#include "kv_cache.cuh"

namespace dspark {

size_t attention_scratch_bytes(int) { return 0; }

namespace {

struct Attention {
    const void *q;
    void *out;
    float *lse;
    long long q_token, q_head, out_token, out_head;
    const int *rows, *cu_new;
    int tokens, q_heads, n_seqs, layer, causal, window;
    float scale;
};

template <typename T, int D>
__global__ void __launch_bounds__(256) attention_kernel(CacheView c, Attention g) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (w >= static_cast<long long>(g.tokens) * g.q_heads) return;
    const int token = static_cast<int>(w / g.q_heads), head = static_cast<int>(w % g.q_heads);
    int s = -1;
    for (int i = 0; i < g.n_seqs; ++i)
        if (g.cu_new[i] <= token && token < g.cu_new[i + 1]) s = i;
    if (s < 0) return;
    const int row = g.rows ? g.rows[s] : s;
    int length = 0;
    if (static_cast<unsigned>(row) < static_cast<unsigned>(c.max_seqs)) {
        length = c.length[row];
        if (length < 0 || length > static_cast<long long>(c.max_pages) * c.page_size) {
            if (lane == 0) atomicOr(c.status, kStatusIndex);
            length = length < 0 ? 0 : c.max_pages * c.page_size;
        }
    } else if (lane == 0) {
        atomicOr(c.status, kStatusIndex);
    }
    const int pos = length - (g.cu_new[s + 1] - token);
    const int end = g.causal ? min(length, pos + 1) : length;
    const int begin = g.window > 0 ? max(0, pos - g.window + 1) : 0;
    const int kv_head = head / (g.q_heads / c.kv_heads);
    const T *q = static_cast<const T *>(g.q) + token * g.q_token + head * g.q_head;
    float x[E], acc[E] = {}, m = -INFINITY, z = 0.f;
    for (int e = 0; e < E; ++e) x[e] = static_cast<float>(q[lane * E + e]) * g.scale;
    const size_t run = size_t(c.page_size) * D;
    for (int j = begin; j < end; ++j) {
        const int page = c.table[size_t(row) * c.max_pages + (j >> c.page_shift)];
        const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(c.num_pages);
        if (!ok && lane == 0) atomicOr(c.status, kStatusIndex);
        const T *k = reinterpret_cast<const T *>(c.pool) +
                     ((size_t(ok ? page : 0) * c.layers + g.layer) * 2 * c.kv_heads + kv_head) * run +
                     size_t(j & (c.page_size - 1)) * D + lane * E;
        const T *v = k + c.kv_heads * run;
        float dot = 0.f;
        for (int e = 0; e < E; ++e) dot += ok ? x[e] * static_cast<float>(k[e]) : 0.f;
        for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        const float up = fmaxf(m, dot), keep = m == -INFINITY ? 0.f : expf(m - up), p = expf(dot - up);
        z = z * keep + p;
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * keep + (ok ? p * static_cast<float>(v[e]) : 0.f);
        m = up;
    }
    T *out = static_cast<T *>(g.out) + token * g.out_token + head * g.out_head;
    for (int e = 0; e < E; ++e) out[lane * E + e] = static_cast<T>(end > begin ? acc[e] / z : 0.f);
    if (g.lse && lane == 0) g.lse[size_t(token) * g.q_heads + head] = end > begin ? m + logf(z) : -INFINITY;
}

}  // namespace

}  // namespace dspark

using namespace dspark;

extern "C" dspark_status dspark_paged_attention(const dspark_cache *cache, int layer, const void *q,
                                                long long q_token_stride, long long q_head_stride, int tokens,
                                                int q_heads, const int32_t *rows, const int32_t *cu_new, int n_seqs,
                                                int max_new, int causal, int window, float scale, void *out,
                                                long long out_token_stride, long long out_head_stride, float *lse,
                                                dspark_stream_t stream) {
    const char *who = "paged_attention";
    CacheView c;
    dspark_status st = cache_view(cache, who, &c);
    if (st != DSPARK_OK) return st;
    if (layer < 0 || layer >= c.layers) return fail(DSPARK_ERR_INVALID, "%s: layer %d of %d", who, layer, c.layers);
    if (tokens < 0 || q_heads < 1 || n_seqs < 0 || max_new < 0 || window < 0)
        return fail(DSPARK_ERR_INVALID, "%s: bad sizes tokens=%d q_heads=%d n_seqs=%d max_new=%d window=%d", who, tokens,
                    q_heads, n_seqs, max_new, window);
    if (q_heads % c.kv_heads) return fail(DSPARK_ERR_INVALID, "%s: %d query heads over %d kv heads", who, q_heads, c.kv_heads);
    if (q_heads / c.kv_heads > 128)
        return fail(DSPARK_ERR_UNSUPPORTED, "%s: %d query heads to a kv head, at most 128", who, q_heads / c.kv_heads);
    if (n_seqs > kMaxSeqs) return fail(DSPARK_ERR_UNSUPPORTED, "%s: n_seqs %d > %d", who, n_seqs, kMaxSeqs);
    if (tokens == 0 || n_seqs == 0) return DSPARK_OK;
    if (!q || !out || !cu_new) return fail(DSPARK_ERR_INVALID, "%s: null pointer argument", who);
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cu_new, 4) || !aligned(lse, 4) || q_token_stride % 8 ||
        q_head_stride % 8 || out_token_stride % 8 || out_head_stride % 8 || q_token_stride < 0 || q_head_stride < 0 ||
        out_token_stride < 0 || out_head_stride < 0)
        return fail(DSPARK_ERR_INVALID, "%s: q and out must be 16-byte aligned, with strides of whole 16 bytes", who);
    Attention g{q, out, lse, q_token_stride, q_head_stride, out_token_stride, out_head_stride, rows, cu_new, tokens, q_heads,
                n_seqs, layer, causal != 0, window, scale};
    const unsigned blocks = static_cast<unsigned>((static_cast<long long>(tokens) * q_heads + 7) / 8);
    const bool bf16 = cache->dtype == DSPARK_BF16;
    if (c.head_dim == 128) {
        if (bf16) attention_kernel<__nv_bfloat16, 128><<<blocks, 256, 0, stream>>>(c, g);
        else attention_kernel<__half, 128><<<blocks, 256, 0, stream>>>(c, g);
    } else {
        if (bf16) attention_kernel<__nv_bfloat16, 64><<<blocks, 256, 0, stream>>>(c, g);
        else attention_kernel<__half, 64><<<blocks, 256, 0, stream>>>(c, g);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DSPARK_OK : cuda_fail(e, who);
}
