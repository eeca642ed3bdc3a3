// Rotary positions: alone (forward and gradient), and on the way into the paged cache.
//
// The angle of pair j at position p is frac(p * turns[j] / 2^64) of a turn.  The product is taken
// modulo 2^64, which drops the whole turns exactly; its top 32 bits, read as a signed fraction of
// half a turn and rounded to fp32, give sine and cosine.  The error of the angle is that rounding, at most 2^-26 of a turn (near
// half a turn, where fp32 has 24 of the 31 bits), whatever the position; p * frequency in fp32 would lose a bit for every
// doubling of the context.
//
// Bound by memory: every element is read and written once.  A block first puts the sines and cosines of its tokens into shared
// memory, one pair to a thread: with every thread computing those of its own unit they took longer than the copies (8190 tokens of
// 40 heads of 128, with the gradient: 82 us at two heads a thread).  Then a thread takes one 32-byte unit of a head (two 16-byte
// vectors that hold whole pairs), three heads at a time; four blocks an SM keep about 100 KB in flight.  That rotation takes
// 57.7 us (5.8 TB/s); appending five prompts of 11,000 tokens of 32 + 8 + 8 heads 45.2 us (6.1 TB/s, 91 % of a copy).
#include "kv_cache.cuh"

namespace dspark {

namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 3;  // heads of a thread in flight
constexpr int kAngles = 2048;  // pairs of a block's tokens: at most kThreads / units tokens of 8 * units pairs

template <typename T> struct Vec;  // 16 bytes of a head
template <> struct Vec<__half> {
    static constexpr int N = 8;
    __device__ static void get(const uint4 &u, float (&f)[8]) {
        const __half2 *h = reinterpret_cast<const __half2 *>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(h[i]);
            f[2 * i] = v.x, f[2 * i + 1] = v.y;
        }
    }
    __device__ static uint4 put(const float (&f)[8]) {
        uint4 u;
        __half2 *h = reinterpret_cast<__half2 *>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        return u;
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static void get(const uint4 &u, float (&f)[8]) {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __bfloat1622float2(h[i]);
            f[2 * i] = v.x, f[2 * i + 1] = v.y;
        }
    }
    __device__ static uint4 put(const float (&f)[8]) {
        uint4 u;
        __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        return u;
    }
};
template <> struct Vec<float> {
    static constexpr int N = 4;
    __device__ static void get(const uint4 &u, float (&f)[4]) {
        f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
    }
    __device__ static uint4 put(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

struct Turns {
    const long long *turns;
    int rotary_dim, layout;
    float amplitude;
    int backward;
};

// Cosine and sine, with the amplitude and the direction, of pair j at a position.
__device__ __forceinline__ float2 angle_of(const Turns &t, int j, int position) {
    const unsigned long long part =
        static_cast<unsigned long long>(static_cast<long long>(position)) * static_cast<unsigned long long>(__ldg(t.turns + j));
    const float x = static_cast<float>(static_cast<int>(part >> 32)) * 0x1p-31f;  // half turns
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(c * t.amplitude, (t.backward ? -s : s) * t.amplitude);
}

// One unit of a head: two 16-byte vectors, half of the turned part (or of the rest) apart, so that neighbouring units are
// neighbouring vectors in either layout; and its pairs' angles.
template <typename T>
struct Unit {
    static constexpr int V = Vec<T>::N;
    int a, b;
    bool turned;
    float cos[V], sin[V];

    __device__ void init(const Turns &t, int unit, int units) {
        const int turning = t.rotary_dim / (2 * V);  // units that are turned
        turned = unit < turning;
        a = turned ? unit * V : t.rotary_dim + (unit - turning) * V;
        b = a + (turned ? turning : units - turning) * V;
    }
    __device__ void take(const float2 *angles, const Turns &t, int unit) {
        if (!turned) return;
        // half: pair i of the unit is (a[i], b[i]); interleaved: the first half of its pairs lie in a, the others in b
        const int first = t.layout == DSPARK_ROTARY_HALF ? unit * V : unit * (V / 2);
        const int second = t.layout == DSPARK_ROTARY_HALF ? first + V / 2 : t.rotary_dim / 4 + first;
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float4 two = *reinterpret_cast<const float4 *>(angles + (i < V / 2 ? first + i : second + i - V / 2));
            cos[i] = two.x, sin[i] = two.y, cos[i + 1] = two.z, sin[i + 1] = two.w;
        }
    }
    __device__ void turn(uint4 &ua, uint4 &ub, int layout) const {
        if (!turned) return;
        float x[V], y[V];
        Vec<T>::get(ua, x);
        Vec<T>::get(ub, y);
        if (layout == DSPARK_ROTARY_HALF) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float p = x[i] * cos[i] - y[i] * sin[i];
                y[i] = y[i] * cos[i] + x[i] * sin[i];
                x[i] = p;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                float p = x[2 * i] * cos[i] - x[2 * i + 1] * sin[i];
                x[2 * i + 1] = x[2 * i + 1] * cos[i] + x[2 * i] * sin[i];
                x[2 * i] = p;
                p = y[2 * i] * cos[V / 2 + i] - y[2 * i + 1] * sin[V / 2 + i];
                y[2 * i + 1] = y[2 * i + 1] * cos[V / 2 + i] + y[2 * i] * sin[V / 2 + i];
                y[2 * i] = p;
            }
        }
        ua = Vec<T>::put(x);
        ub = Vec<T>::put(y);
    }
};

struct Strided {
    const void *p;
    long long token, head;
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(Strided x, Strided y, int tokens, int heads, int units,
                                                          int lanes, const int *positions, Turns t) {
    __shared__ __align__(16) float2 s_angles[kAngles];
    pdl_launch_dependents();
    pdl_wait();
    // units * lanes threads to a token: `lanes` heads at a time
    const int per = units * lanes, count = kThreads / per, half = t.rotary_dim / 2;
    const int token0 = static_cast<int>(blockIdx.x) * count, here = min(count, tokens - token0);
    for (int i = threadIdx.x; i < here * half; i += kThreads) {
        const int k = i / half;
        s_angles[i] = angle_of(t, i - k * half, positions[token0 + k]);
    }
    __syncthreads();
    const int k = static_cast<int>(threadIdx.x) / per, token = token0 + k;
    if (k >= here) return;
    const int r = threadIdx.x % per, unit = r % units;
    Unit<T> u;
    u.init(t, unit, units);
    u.take(s_angles + k * half, t, unit);
    const T *px = static_cast<const T *>(x.p) + token * x.token;
    T *py = static_cast<T *>(const_cast<void *>(y.p)) + token * y.token;
    const int step = lanes * static_cast<int>(gridDim.y);
    for (int h0 = r / units + static_cast<int>(blockIdx.y) * lanes; h0 < heads; h0 += kHeads * step) {
        uint4 a[kHeads], b[kHeads];
#pragma unroll
        for (int q = 0; q < kHeads; ++q) {
            const int h = h0 + q * step;
            if (h < heads) {
                a[q] = *reinterpret_cast<const uint4 *>(px + h * x.head + u.a);
                b[q] = *reinterpret_cast<const uint4 *>(px + h * x.head + u.b);
            }
        }
#pragma unroll
        for (int q = 0; q < kHeads; ++q) {
            const int h = h0 + q * step;
            if (h < heads) {
                u.turn(a[q], b[q], t.layout);
                *reinterpret_cast<uint4 *>(py + h * y.head + u.a) = a[q];
                *reinterpret_cast<uint4 *>(py + h * y.head + u.b) = b[q];
            }
        }
    }
}

struct Append {
    Strided q, k, v, out;
    const int *rows, *cu_new, *positions;
    int tokens, q_heads, n_seqs, layer;
};

// Sequence of token t: the last s with cu_new[s] <= t; -1 outside all of them.  One warp.
__device__ int sequence_of(const int *cu, int n_seqs, int t, int lane) {
    int at_or_before = 0;
    for (int s0 = 0; s0 <= n_seqs; s0 += 32) {
        const int s = s0 + lane;
        at_or_before += __popc(__ballot_sync(0xffffffffu, s <= n_seqs && cu[s] <= t));
    }
    return at_or_before >= 1 && at_or_before <= n_seqs ? at_or_before - 1 : -1;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(CacheView c, Append g, int units, int lanes, Turns t) {
    __shared__ int s_pos[kThreads / 4];        // angle's position of each token of the block
    __shared__ __align__(16) float2 s_angles[kAngles];
    __shared__ long long s_slot[kThreads / 4]; // element of the pool where its first key goes; -1: nowhere; -2: no token
    pdl_launch_dependents();
    pdl_wait();
    const int per = units * lanes, count = kThreads / per;
    const int token0 = static_cast<int>(blockIdx.x) * count, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long run = static_cast<long long>(c.page_size) * c.head_dim;  // elements of one (page, layer, k or v, head)
    for (int i = warp; i < count; i += kThreads / 32) {
        const int token = token0 + i;
        const int s = token < g.tokens ? sequence_of(g.cu_new, g.n_seqs, token, lane) : -1;
        if (lane != 0) continue;
        long long slot = -2;
        int pos = 0;
        if (s >= 0) {
            const int row = g.rows ? g.rows[s] : s;
            slot = -1;
            if (static_cast<unsigned>(row) < static_cast<unsigned>(c.max_seqs)) {
                pos = c.length[row] - g.cu_new[s + 1] + token;
                const int j = pos >> c.page_shift;
                if (pos >= 0 && j < c.max_pages) {
                    const int page = c.table[static_cast<size_t>(row) * c.max_pages + j];
                    if (static_cast<unsigned>(page) < static_cast<unsigned>(c.num_pages))
                        slot = (static_cast<long long>(page) * c.layers + g.layer) * 2 * c.kv_heads * run +
                               static_cast<long long>(pos & (c.page_size - 1)) * c.head_dim;
                }
            }
            if (slot < 0 && blockIdx.y == 0) atomicOr(c.status, kStatusIndex);
            if (g.positions) pos = g.positions[token];
        }
        s_pos[i] = pos;
        s_slot[i] = slot;
    }
    __syncthreads();
    const int half = t.rotary_dim / 2;
    for (int a = threadIdx.x; a < count * half; a += kThreads) {
        const int k = a / half;
        if (s_slot[k] != -2) s_angles[a] = angle_of(t, a - k * half, s_pos[k]);
    }
    __syncthreads();
    const int i = threadIdx.x / per;
    if (i >= count) return;
    const long long slot = s_slot[i];
    if (slot == -2) return;
    const long long token = token0 + i;
    const int r = threadIdx.x % per, unit = r % units;
    Unit<T> u;
    u.init(t, unit, units);
    u.take(s_angles + i * half, t, unit);
    const int heads = g.q_heads + 2 * c.kv_heads;
    T *pool = reinterpret_cast<T *>(c.pool);
    const int step = lanes * static_cast<int>(gridDim.y);
    for (int h0 = r / units + static_cast<int>(blockIdx.y) * lanes; h0 < heads; h0 += kHeads * step) {
        uint4 a[kHeads], b[kHeads];
#pragma unroll
        for (int q = 0; q < kHeads; ++q) {
            const int h = h0 + q * step, hk = h - g.q_heads, hv = hk - c.kv_heads;
            if (h < heads) {
                const Strided &from = hk < 0 ? g.q : hv < 0 ? g.k : g.v;
                const T *px = static_cast<const T *>(from.p) + token * from.token + (hk < 0 ? h : hv < 0 ? hk : hv) * from.head;
                a[q] = *reinterpret_cast<const uint4 *>(px + u.a);
                b[q] = *reinterpret_cast<const uint4 *>(px + u.b);
            }
        }
#pragma unroll
        for (int q = 0; q < kHeads; ++q) {
            const int h = h0 + q * step, hk = h - g.q_heads, hv = hk - c.kv_heads;
            if (h < heads && (hk < 0 || slot >= 0)) {
                if (hv < 0) u.turn(a[q], b[q], t.layout);
                // a layer's runs of a page: the kv_heads of k, then those of v
                T *py = hk < 0 ? static_cast<T *>(const_cast<void *>(g.out.p)) + token * g.out.token + h * g.out.head : pool + slot + hk * run;
                *reinterpret_cast<uint4 *>(py + u.a) = a[q];
                *reinterpret_cast<uint4 *>(py + u.b) = b[q];
            }
        }
    }
}

// The threads of a token: `units` of them for each of `lanes` heads at a time.  With many tokens eight heads at a time: four tokens of
// 128-element heads to a block, over which its lookups and angles are spread.  With few, more, until there are 512 threads an SM.
void shape(int tokens, int heads, int units, int sms, int *lanes, int *blocks_x, int *blocks_y) {
    int l = 8;
    while (2 * l * units <= kThreads && l < heads && static_cast<long long>(tokens) * units * l < 512ll * sms) l *= 2;
    if (l > heads) l = heads;
    if (l > kThreads / units) l = kThreads / units;
    const int each = static_cast<long long>(tokens) * units * l >= 512ll * sms ? (heads + l - 1) / l : 1;  // heads of a thread
    const int count = kThreads / (units * l);
    *lanes = l;
    *blocks_x = (tokens + count - 1) / count;
    *blocks_y = (heads + l * each - 1) / (l * each);
}

int element_bytes(int dtype) { return dtype == DSPARK_FP32 ? 4 : 2; }

dspark_status check_turns(const char *who, const int64_t *turns, int rotary_dim, int layout, int head_dim) {
    if (layout != DSPARK_ROTARY_HALF && layout != DSPARK_ROTARY_INTERLEAVED)
        return fail(DSPARK_ERR_INVALID, "%s: layout %d", who, layout);
    if (rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16)
        return fail(DSPARK_ERR_UNSUPPORTED, "%s: rotary_dim %d (a multiple of 16 up to head_dim %d)", who, rotary_dim, head_dim);
    if (!turns || !aligned(turns, 8)) return fail(DSPARK_ERR_INVALID, "%s: turns must be an 8-byte aligned array", who);
    return DSPARK_OK;
}

// Also drops the strides of axes of one entry: nothing moves along them, and tensors come with any value there.
dspark_status check_strided(const char *who, const char *name, Strided *s, int tokens, int heads, int bytes) {
    if (!s->p) return fail(DSPARK_ERR_INVALID, "%s: null pointer argument (%s)", who, name);
    if (tokens == 1) s->token = 0;
    if (heads == 1) s->head = 0;
    if (!aligned(s->p, 16) || s->token * bytes % 16 || s->head * bytes % 16 || s->token < 0 || s->head < 0)
        return fail(DSPARK_ERR_INVALID, "%s: %s must be 16-byte aligned, with strides of whole 16 bytes (%lld, %lld)", who, name,
                    s->token, s->head);
    return DSPARK_OK;
}

}  // namespace

}  // namespace dspark

using namespace dspark;

extern "C" dspark_status dspark_rotary(const dspark_rotary_args *args, dspark_stream_t stream) {
    clear_error();
    if (!args) return fail(DSPARK_ERR_INVALID, "rotary: null arguments");
    const auto [x, y, positions, turns, x_token_stride, x_head_stride, y_token_stride, y_head_stride, dtype, tokens, heads, head_dim,
                rotary_dim, layout, backward, amplitude] = *args;
    if (dtype != DSPARK_FP16 && dtype != DSPARK_BF16 && dtype != DSPARK_FP32)
        return fail(DSPARK_ERR_INVALID, "rotary: dtype %d", dtype);
    if (tokens < 0 || heads < 0) return fail(DSPARK_ERR_INVALID, "rotary: bad sizes tokens=%d heads=%d", tokens, heads);
    if (head_dim < 16 || head_dim > 512 || head_dim % 16)
        return fail(DSPARK_ERR_UNSUPPORTED, "rotary: head_dim %d (a multiple of 16 up to 512)", head_dim);
    dspark_status st = check_turns("rotary", turns, rotary_dim, layout, head_dim);
    if (st != DSPARK_OK || tokens == 0 || heads == 0) return st;
    const int bytes = element_bytes(dtype);
    Strided sx{x, x_token_stride, x_head_stride}, sy{y, y_token_stride, y_head_stride};
    if ((st = check_strided("rotary", "x", &sx, tokens, heads, bytes)) != DSPARK_OK) return st;
    if ((st = check_strided("rotary", "y", &sy, tokens, heads, bytes)) != DSPARK_OK) return st;
    if (!positions || !aligned(positions, 4)) return fail(DSPARK_ERR_INVALID, "rotary: positions must be a 4-byte aligned array");
    int sms = 0;
    if ((st = static_cast<dspark_status>(current_sm_count(&sms))) != DSPARK_OK) return st;
    const int units = head_dim * bytes / 32;
    int lanes, bx, by;
    shape(tokens, heads, units, sms, &lanes, &bx, &by);
    const Turns t{reinterpret_cast<const long long *>(turns), rotary_dim, layout, amplitude, backward != 0};
    const dim3 grid(bx, by);
    auto *kernel = dtype == DSPARK_FP32 ? rotary_kernel<float> : dtype == DSPARK_BF16 ? rotary_kernel<__nv_bfloat16> : rotary_kernel<__half>;
    const cudaError_t e = launch_pdl(kernel, grid, dim3(kThreads), 0, stream, sx, sy, tokens, heads, units, lanes, positions, t);
    return e == cudaSuccess ? DSPARK_OK : cuda_fail(e, "rotary");
}

extern "C" dspark_status dspark_rotary_append(const dspark_cache *cache, const dspark_append_args *args, dspark_stream_t stream) {
    const char *who = "rotary_append";
    CacheView c;
    dspark_status st = cache_view(cache, who, &c);
    if (st != DSPARK_OK) return st;
    if (!args) return fail(DSPARK_ERR_INVALID, "%s: null arguments", who);
    const auto [q, k, v, q_out, rows, cu_new, positions, turns, q_token_stride, q_head_stride, k_token_stride, k_head_stride,
                v_token_stride, v_head_stride, out_token_stride, out_head_stride, layer, tokens, q_heads, n_seqs, rotary_dim, layout,
                amplitude] = *args;
    if (layer < 0 || layer >= c.layers) return fail(DSPARK_ERR_INVALID, "%s: layer %d of %d", who, layer, c.layers);
    if (tokens < 0 || q_heads < 0 || n_seqs < 0)
        return fail(DSPARK_ERR_INVALID, "%s: bad sizes tokens=%d q_heads=%d n_seqs=%d", who, tokens, q_heads, n_seqs);
    if (n_seqs > kMaxSeqs) return fail(DSPARK_ERR_UNSUPPORTED, "%s: n_seqs %d > %d", who, n_seqs, kMaxSeqs);
    if ((st = check_turns(who, turns, rotary_dim, layout, c.head_dim)) != DSPARK_OK || tokens == 0 || n_seqs == 0) return st;
    Append g;
    g.q = Strided{q, q_token_stride, q_head_stride};
    g.k = Strided{k, k_token_stride, k_head_stride};
    g.v = Strided{v, v_token_stride, v_head_stride};
    g.out = Strided{q_out, out_token_stride, out_head_stride};
    if (q_heads > 0) {
        if ((st = check_strided(who, "q", &g.q, tokens, q_heads, 2)) != DSPARK_OK) return st;
        if ((st = check_strided(who, "q_out", &g.out, tokens, q_heads, 2)) != DSPARK_OK) return st;
    }
    if ((st = check_strided(who, "k", &g.k, tokens, c.kv_heads, 2)) != DSPARK_OK) return st;
    if ((st = check_strided(who, "v", &g.v, tokens, c.kv_heads, 2)) != DSPARK_OK) return st;
    if (!cu_new || !aligned(cu_new, 4)) return fail(DSPARK_ERR_INVALID, "%s: cu_new must be a 4-byte aligned array", who);
    int sms = 0;
    if ((st = static_cast<dspark_status>(current_sm_count(&sms))) != DSPARK_OK) return st;
    const int units = c.head_dim * 2 / 32;
    int lanes, bx, by;
    shape(tokens, q_heads + 2 * c.kv_heads, units, sms, &lanes, &bx, &by);
    const Turns t{reinterpret_cast<const long long *>(turns), rotary_dim, layout, amplitude, 0};
    g.rows = rows;
    g.cu_new = cu_new;
    g.positions = positions;
    g.tokens = tokens;
    g.q_heads = q_heads;
    g.n_seqs = n_seqs;
    g.layer = layer;
    auto *kernel = cache->dtype == DSPARK_BF16 ? append_kernel<__nv_bfloat16> : append_kernel<__half>;
    const cudaError_t e = launch_pdl(kernel, dim3(bx, by), dim3(kThreads), 0, stream, c, g, units, lanes, t);
    return e == cudaSuccess ? DSPARK_OK : cuda_fail(e, who);
}
