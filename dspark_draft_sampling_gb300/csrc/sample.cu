// Drawing tokens from logits (temperature, top-k, top-p, min-p), and judging drafted tokens against the target's logits.
//
// Weights.  A row's token v weighs w_v = exp((l_v - m) / T), m the largest logit.  Sums over a vocabulary decide which token a
// uniform number falls on and where a nucleus ends, so they have to come out the same each time they are taken, in whatever order blocks and
// warps add: weights are whole numbers of 2^-44, sums 64-bit integers; only light tokens of 32 bytes are added in 32-bit floating point
// first, in one order (2^-21 of what they weigh at most), and cut to whole units together; a draw that falls on them looks at their terms
// uncut.  With y = (l - m) log2(e) / T in two 32-bit parts, 2^y of the tokens that matter (y >= -6) comes
// from a table of 2^(j/64) and a cubic in the rest |r| <= 2^-7, whose next term is 4e-11: 28 bits.  Lighter tokens take the fast
// exponential (2^-22) of a difference rounded to 32 bits (2^-24 of |ln w|): 2^-27 of the heaviest token's weight at most.
//
// Work.  A row belongs to a cluster of thread blocks, each of which keeps its slice in shared memory, so the logits are read from
// memory once whatever the settings ask for.  The blocks exchange maxima, sums and histograms through distributed shared memory, at 1 to 1.5
// microseconds an exchange (the cluster's barrier and the wait for the slowest block).  What is decided by what was exchanged is the same in
// all blocks, so that they meet at the same barriers.
//
// Measured (GB300).  256 rows of 248320 bf16, nothing dropped: 65 us, 2.0 TB/s (the bytes alone 19); 8 x 15 drafts of 248320 fp32 79 us; 96
// rows of 151936 bf16 whose nuclei hold 75,000 tokens 120 us; 28 of fp32 with nuclei of 20,000 and their distributions 45; one row with top-k
// 50 10, of which 2.5 are the launch; one request's seven drafts, nuclei of a few to 20,000 tokens, 24 to 29.  Blocks wait at barriers for most of
// the time that is not instructions (44 to 60 % of the issue slots are used).
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstring>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace dspark {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBinBits = 9, kBins = 1 << kBinBits;  // of a histogram
static_assert(kBins == kThreads, "a thread looks after a bin");
constexpr int kOctave = kBins / 64;       // of them to a power of two, where they divide weights
constexpr float kSpread = kBins - 0.1f;   // bins of equal width over a range, short of the end
constexpr int kList = kThreads;           // tokens that one block sorts: a thread to each
constexpr int kNear = 1024;               // tokens of a block's slice around a nucleus' end
constexpr int kMaxBlocks = 16;            // of a cluster
constexpr int kMostSlice = 128 * 1024;    // bytes; 2^19 fp32 logits over kMaxBlocks blocks
static_assert(kMostSlice / (kThreads * 32) + 1 <= kWarps, "a slice's rounds of 32 bytes a thread are one for each warp at most");
constexpr int kHeavy = 6;                 // powers of two below the heaviest token down to which weights are exact to 28 bits
constexpr int kCounted = 10;               // powers of two below it down to which a nucleus' end is looked for among all tokens
constexpr float kLowest = -3.402823466e38f;
constexpr int kNoIndex = -0x7fffffff;      // before all indices, also those of what pads a slice
constexpr int kMaxVocab = 1 << 19;        // 2^19 weights of 2^44 stay below 2^64
constexpr long long kAccepted = -2;       // in ids until the second kernel has run: the row's draft is accepted

using u64 = unsigned long long;

struct Draw {
    const void *logits;
    const float *uniforms, *temperature, *top_p, *min_p, *draft_probs;
    const int *top_k, *cu_drafts;
    const long long *drafts;
    long long *ids;
    int *accepted;
    float *probs;
    long long logits_stride, probs_stride, draft_probs_stride;
    float temperature_all, top_p_all, min_p_all;
    int top_k_all;
    float floor_hi_all, floor_lo_all;  // log2(min_p_all)
    int rows, vocab, slice, n_seqs, n_drafts;
    uint2 table[64];  // 2^(28 + j/64): rounded, and as a float
};

// What a row is drawn by: the cluster's first block reads it and hands it to the others, so that all of them take the same branches
// whatever happens to those arrays meanwhile.
struct Given {
    float hi, lo, least;       // log2(e) / T in two parts; a difference of logits whose weight is 0
    float floor_hi, floor_lo;  // log2 of min_p
    float top_p, u;
    int top_k;                 // 0: all
    int state;                 // one of the below
    int token;                 // the draft that the row judges; -1: none that can be accepted
    float logit, share, accept;  // its logit, its probability when it was drawn, the number that decides
    int draft;                 // its place among all drafts
};
enum { kNotDrawn, kGreedy, kDrawn };

struct alignas(16) Shared {
    uint2 table[64];
    Given given;
    int found, to_bin, from_bin, likely, least_from;
    float share_hi, share_lo;    // what turns a light weight into a probability
    float at_low[2], at_high[2], at_to, at_from, at_likely;
    unsigned listed, nears, heavies;
    u64 slot[2][3][kMaxBlocks];  // [parity][value][block]: what the blocks exchange
    u64 said[2][4];              // [parity][value]: what the first warp makes of it
    u64 warp[kWarps];            // sums over the warps' stretches of the slice
    u64 scan[2][kWarps];
    u64 inverse, last;           // last: of the kept tokens, as in the list
    u64 z, drafted;
    u64 count_before, mass_before, count_in;
    // from here on not used, and not there, where nothing is dropped
    alignas(16) unsigned count[2][kBins];  // histograms, read by the cluster's other blocks
    union {                      // lists are sorted when all blocks have done with the last histogram
        unsigned mass[2][kBins][2];  // low and high half of 64 bits
        u64 sort[2][kList];
    };
    u64 all_mass[kBins];         // of all blocks
    unsigned all_count[kBins];
    u64 list[kList];             // this block's tokens of a list, read by the first block: order code and what is left of 2^32 behind the index
    u64 near_end[kNear];         // tokens near a nucleus' end in the same form, this block's own
};

constexpr size_t shared_bytes(bool whole) { return whole ? offsetof(Shared, count) : sizeof(Shared); }
static_assert(offsetof(Shared, mass) % 8 == 0 && offsetof(Shared, slot) % 8 == 0 && shared_bytes(true) % 16 == 0 && shared_bytes(false) % 16 == 0,
              "64-bit words and vectors are aligned");

__device__ __forceinline__ uint32_t at_block(const void *p, int block) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(block));
    return r;
}
__device__ __forceinline__ unsigned ld_block_u32(uint32_t at) {
    unsigned v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ u64 ld_block_u64(uint32_t at) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void st_block_u32(uint32_t at, unsigned v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void st_block_u64(uint32_t at, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}
// Every thread of the cluster; orders their memory accesses.
__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The logit of an order code in the upper half.
__device__ __forceinline__ float value_of(u64 key) {
    const unsigned c = static_cast<unsigned>(key >> 32);
    return __uint_as_float(c & 0x80000000u ? c & 0x7fffffffu : ~c);
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <typename N>
__device__ __forceinline__ N warp_prefix(N v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const N y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// floor(z * f), or its ceiling, exactly; f in [0, 1).
__device__ __forceinline__ u64 part_of(u64 z, float f, bool up) {
    const unsigned bits = __float_as_uint(f), mantissa = (bits & 0x7fffffu) | (bits >> 23 ? 0x800000u : 0u);
    const unsigned shift = 150 - max(bits >> 23, 1u);  // 24 to 149
    const u64 high = __umul64hi(z, mantissa), low = z * mantissa;
    u64 whole = 0, rest = high | low;
    if (shift < 64) {
        whole = high << (64 - shift) | low >> shift;
        rest = low << (64 - shift);
    } else if (shift < 128) {
        whole = high >> (shift - 64);
        rest = low | (high & ((1ull << (shift - 64)) - 1));
    }
    return whole + (up && rest != 0 ? 1 : 0);
}

// Where a uniform number falls among z.
__device__ __forceinline__ u64 place_of(float u, u64 z) { return !(u > 0.f) ? 0 : u < 1.f ? part_of(z, u, false) : z - 1; }

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16 bytes of logits of a type.
template <typename T>
struct Type;
template <>
struct Type<float> {
    static constexpr int kVector = 4, kPer = 2 * kVector;  // tokens of 16 bytes, and of the 32 that a thread takes at a time
    static constexpr unsigned kMasked = 0xff800000u;  // -infinity
    static __device__ __forceinline__ void spread(uint4 v, float *x) {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float one(const void *p, long long i) { return static_cast<const float *>(p)[i]; }
    // The larger ones of two vectors, and the largest of one, NaN left aside.
    static __device__ __forceinline__ uint4 larger(uint4 a, uint4 b) {
        auto most = [](unsigned x, unsigned y) { return __float_as_uint(fmaxf(__uint_as_float(x), __uint_as_float(y))); };
        return make_uint4(most(a.x, b.x), most(a.y, b.y), most(a.z, b.z), most(a.w, b.w));
    }
    static __device__ __forceinline__ float largest(uint4 v) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    // One value throughout, rounded down; that value; about the lowest one.
    static __device__ __forceinline__ unsigned down(float x) { return __float_as_uint(x); }
    static __device__ __forceinline__ float low(unsigned v) { return __uint_as_float(v); }
    static constexpr float kLeast = -3.0e38f;
    static constexpr bool kFine = true;
};
template <>
struct Type<__nv_bfloat16> {
    static constexpr int kVector = 8, kPer = 2 * kVector;
    static constexpr unsigned kMasked = 0xff80ff80u;
    static __device__ __forceinline__ void spread(uint4 v, float *x) {
        const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    static __device__ __forceinline__ float one(const void *p, long long i) {
        return __uint_as_float(static_cast<unsigned>(static_cast<const unsigned short *>(p)[i]) << 16);
    }
    static __device__ __forceinline__ unsigned most(unsigned a, unsigned b) {
        unsigned r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint4 larger(uint4 a, uint4 b) { return make_uint4(most(a.x, b.x), most(a.y, b.y), most(a.z, b.z), most(a.w, b.w)); }
    static __device__ __forceinline__ float largest(uint4 v) {
        const unsigned m = most(most(v.x, v.y), most(v.z, v.w));
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
    static __device__ __forceinline__ unsigned down(float x) {
        const unsigned b = __float_as_uint(x), up = (b & 0x80000000u ? b + 0xffffu : b) >> 16;
        return up | up << 16;
    }
    static __device__ __forceinline__ float low(unsigned v) { return __uint_as_float(v << 16); }
    static constexpr float kLeast = -3.0e38f;
    static constexpr bool kFine = false;  // differences of 8-bit significands are exact but for the smallest logits'
};
template <>
struct Type<__half> {
    static constexpr int kVector = 8, kPer = 2 * kVector;
    static constexpr unsigned kMasked = 0xfc00fc00u;
    static __device__ __forceinline__ void spread(uint4 v, float *x) {
        const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ float one(const void *p, long long i) { return __half2float(static_cast<const __half *>(p)[i]); }
    static __device__ __forceinline__ unsigned most(unsigned a, unsigned b) {
        unsigned r;
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint4 larger(uint4 a, uint4 b) { return make_uint4(most(a.x, b.x), most(a.y, b.y), most(a.z, b.z), most(a.w, b.w)); }
    static __device__ __forceinline__ float largest(uint4 v) {
        const unsigned m = most(most(v.x, v.y), most(v.z, v.w));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&m));
        return fmaxf(f.x, f.y);
    }
    static __device__ __forceinline__ unsigned down(float x) {
        const unsigned h = __half_as_ushort(__float2half_rd(x));
        return h | h << 16;
    }
    static __device__ __forceinline__ float low(unsigned v) { return __half2float(__ushort_as_half(static_cast<unsigned short>(v))); }
    static constexpr float kLeast = -6.0e4f;
    static constexpr bool kFine = true;
};

// A number of 0 to 2^63 rounded down, by shifts: the conversion instruction runs at the rate of 64-bit floating point, 15 cycles a warp.
__device__ __forceinline__ u64 to_whole(float x) {
    const unsigned bits = __float_as_uint(x);
    const int shift = static_cast<int>(bits >> 23) - 150;
    const u64 m = (bits & 0x7fffffu) | 0x800000u;
    return shift >= 0 ? m << shift : shift > -24 ? m >> -shift : 0;
}

// The weights of a row's tokens.
template <typename T>
struct Weights {
    float top, hi, lo, least;   // m; log2(e) / T in two parts; a difference of logits whose weight is 0
    unsigned clamp;             // a logit of that difference or a larger one, in the logits' type
    bool simple;                // whether there is one that weighs nothing and leaves all numbers finite
    const uint2 *table;

    __device__ __forceinline__ Weights(float m, const Given &g, const uint2 *t) : top(m), hi(g.hi), lo(g.lo), least(g.least), table(t) {
        clamp = Type<T>::down(top + least);
        const float y = (Type<T>::low(clamp) - top) * hi;
        simple = y <= -127.f && y > -1.0e4f && top + least > Type<T>::kLeast && top < 1.0e37f;  // 2^y is flushed to 0
    }
    // y of a logit that is not NaN, as two parts
    __device__ __forceinline__ void exponent(float l, float *p, float *e) const {
        const float diff = l - top, d = l >= top ? 0.f : fmaxf(diff, least);
        *p = d * hi;
        *e = __fmaf_rn(d, lo, __fmaf_rn(d, hi, -*p));
        if ((heavy(*p) || Type<T>::kFine) && d < 0.f && d > least) {  // and what the difference lost
            const float back = diff - l, lost = (l - (diff - back)) + (-top - back);
            *e = __fmaf_rn(lost, hi, *e);
        }
    }
    __device__ __forceinline__ static bool heavy(float p) { return p >= -static_cast<float>(kHeavy); }
    // 2^(28 + fraction) in whole numbers and the power of two that it is to be divided by
    __device__ __forceinline__ unsigned significand(float p, float e, int *shift) const { return significand(p, e, table, shift); }
    __device__ __forceinline__ static unsigned significand(float p, float e, const uint2 *table, int *shift) {
        const float t = p + 196608.f;  // 1.5 * 2^17: rounded to 64ths
        const int n = __float_as_int(t) - 0x48400000;
        const float r = (p - (t - 196608.f)) + e;
        const float q = r * __fmaf_rn(r, __fmaf_rn(r, 0.0555041087f, 0.2402265070f), 0.6931471806f);
        const uint2 entry = table[n & 63];
        *shift = -(n >> 6);
        return entry.x + (__float_as_int(__fmaf_rn(q, __uint_as_float(entry.y), 12582912.f)) - 0x4b400000);
    }
    __device__ __forceinline__ u64 heavy_weight(float p, float e) const {
        int shift;
        const unsigned s = significand(p, e, &shift);
        return static_cast<u64>(s) << (16 - shift);
    }
    __device__ __forceinline__ static float light_weight(float p, float e) {  // of 2^-44
        const float w = fast_exp2(p) * 0x1p44f;
        return __fmaf_rn(w * 0.6931471806f, e, w);
    }
    // Light weights in whole numbers. The fast exponential falls short by 5.1e-8 on average (rms 5.9e-8, at most 1.42e-7, over -40..-8 on
    // this GPU), which would shift light tokens against heavy ones: 2^-24 is added back.
    __device__ __forceinline__ static u64 whole(float c) {
        const u64 v = to_whole(c);
        return v + (v >> 24);
    }
    __device__ __forceinline__ u64 weight(float l) const {
        float p, e;
        exponent(l, &p, &e);
        return heavy(p) ? heavy_weight(p, e) : whole(light_weight(p, e));
    }
};

// Which tokens are left: those before and with the last one of the order.
struct Kept {
    float value;  // the last token's logit, and the last index of its ties that stays
    int index;

    __device__ __forceinline__ bool order(float l, int i) const { return l > value || (l == value && i <= index); }
};

// take(u, weights of tokens 2u and 2u + 1) for a vector's light tokens, in 32 bits and units of the heaviest one: some 10 instructions a token where the
// general form takes 40 and more. 0 (or not called) for those that are not kept, and for the ones whose bits are returned: tokens that are not light, or
// as large as the last kept one, of which indices decide. They are few, and looked at one by one.
template <typename T, typename F>
__device__ __forceinline__ unsigned light_weights(const Weights<T> &w, const Kept &kept, const uint4 *at, F take) {
    constexpr int P = Type<T>::kPer;
    const uint4 v0 = at[0], v1 = at[1];
    const float most = Type<T>::largest(Type<T>::larger(v0, v1));
    if (most < kept.value || !w.simple) return w.simple ? 0u : (1u << P) - 1u;
    const uint4 c = make_uint4(w.clamp, w.clamp, w.clamp, w.clamp);
    float x[P];
    Type<T>::spread(Type<T>::larger(v0, c), x);  // also from NaN and -infinity
    Type<T>::spread(Type<T>::larger(v1, c), x + P / 2);
    unsigned special = 0;
    if (w.heavy((most - w.top) * w.hi)) {
        const float none = w.top + w.least;
#pragma unroll
        for (int u = 0; u < P; ++u)
            if (w.heavy((x[u] - w.top) * w.hi)) {
                special |= 1u << u;
                x[u] = none;
            }
    }
    if (kept.value > -INFINITY) {
        const float none = w.top + w.least;
#pragma unroll
        for (int u = 0; u < P; ++u) {
            if (x[u] == kept.value) special |= 1u << u;
            x[u] = x[u] > kept.value ? x[u] : none;
        }
    }
    const u64 top = pair_f32(-w.top, -w.top), hi = pair_f32(w.hi, w.hi), less_hi = pair_f32(-w.hi, -w.hi), less_lo = pair_f32(-w.lo, -w.lo),
              less_ln2 = pair_f32(-0.6931471806f, -0.6931471806f), back = pair_f32(w.top, w.top), minus = pair_f32(-1.f, -1.f);
#pragma unroll
    for (int u = 0; u < P / 2; ++u) {
        const u64 d = add_f32x2(pair_f32(x[2 * u], x[2 * u + 1]), top), p = mul_f32x2(d, hi);
        u64 e = fma_f32x2(d, less_lo, fma_f32x2(d, less_hi, p));  // what p lacks, negative
        if (Type<T>::kFine)  // and what the difference lost: that of 24 bits, or of small logits, is not exact
            e = fma_f32x2(fma_f32x2(add_f32x2(d, back), minus, pair_f32(x[2 * u], x[2 * u + 1])), less_hi, e);
        float a, b;
        split_f32(p, &a, &b);
        const u64 two = pair_f32(fast_exp2(a), fast_exp2(b));
        take(u, fma_f32x2(mul_f32x2(two, less_ln2), e, two));
    }
    return special;
}

// Sums over a vector's tokens, in index order: the sum up to a token never falls, and the sum over the vector is the same whenever it is
// taken.
template <typename T, bool SKIP = false>
struct MassSum {
    const Weights<T> &w;
    const Kept &kept;
    int skip;  // a token left out
    u64 h = 0;
    float c = 0.f;
    __device__ __forceinline__ MassSum(const Weights<T> &a, const Kept &b, int without = -1) : w(a), kept(b), skip(without) {}
    __device__ __forceinline__ void add(float l, int i) {
        if (!kept.order(l, i) || (SKIP && i == skip)) return;
        float p, e;
        w.exponent(l, &p, &e);
        if (w.heavy(p)) h += w.heavy_weight(p, e);
        else c += w.light_weight(p, e);
    }
    __device__ __forceinline__ u64 sum() const { return h + w.whole(c); }
    __device__ __forceinline__ static u64 up(float x) {  // light weights in whole numbers, rounded up
        const u64 v = to_whole(x);
        return v + (v >> 24) + (static_cast<float>(v) < x ? 1 : 0);
    }
    // What token t of a vector adds to vector(), in h and c.
    __device__ __forceinline__ void token(const uint4 *at, int first, int t) {
        const unsigned special = light_weights(w, kept, at, [&](int u, u64 two) {
            float a, b;
            split_f32(two, &a, &b);
            if (u == t >> 1) c = (t & 1 ? b : a) * 0x1p44f;
        });
        if (SKIP && first + t == skip) c = 0.f;
        if (special >> t & 1) add(Type<T>::one(at, t), first + t);
    }
    __device__ __forceinline__ u64 vector(const uint4 *at, int first) {
        constexpr int P = Type<T>::kPer;
        u64 s[2] = {0, 0};
        const bool skips = static_cast<unsigned>(skip - first) < P;
        unsigned special = light_weights(w, kept, at, [&](int u, u64 two) {
            if (SKIP && skips && (skip - first) >> 1 == u) {
                float a, b;
                split_f32(two, &a, &b);
                two = (skip - first) & 1 ? pair_f32(a, 0.f) : pair_f32(0.f, b);
            }
            s[u & 1] = add_f32x2(s[u & 1], two);
        });
        float a, b;
        split_f32(add_f32x2(s[0], s[1]), &a, &b);
        c = (a + b) * 0x1p44f;
        for (; special; special &= special - 1) {
            const int u = __ffs(special) - 1;
            add(Type<T>::one(at, u), first + u);
        }
        return sum();
    }
};

template <typename T>
struct TieSum {
    float value;
    const Kept &kept;
    u64 h = 0;
    static constexpr float c = 0.f;
    __device__ __forceinline__ TieSum(float v, const Kept &b) : value(v), kept(b) {}
    __device__ __forceinline__ void add(float l, int i) { h += l == value && kept.order(l, i) ? 1 : 0; }
    __device__ __forceinline__ static u64 up(float) { return 0; }
    __device__ __forceinline__ void token(const uint4 *at, int first, int t) { add(Type<T>::one(at, t), first + t); }
    __device__ __forceinline__ u64 vector(const uint4 *at, int first) {
        float x[Type<T>::kPer];
        Type<T>::spread(at[0], x);
        Type<T>::spread(at[1], x + Type<T>::kVector);
#pragma unroll
        for (int u = 0; u < Type<T>::kPer; ++u) add(x[u], first + u);
        return h;
    }
};

// Leading zeros of a row's sum: 0 to 19, as 2^44 <= z.
__device__ __forceinline__ int lead_of(u64 z) { return __clzll(static_cast<long long>(z)); }

// max(0, p - q) in 2^-62 over the kept tokens. Of light ones p and the difference are taken in 32 bits, p with a share in two parts.
template <typename T>
struct RestSum {
    const Weights<T> &w;
    const Kept &kept;
    const float *q;
    int vocab, shift;
    u64 inverse;
    float share_hi, share_lo;
    u64 h = 0;
    float c = 0.f;
    // What p is taken by, of the row's sum z: 2^127 / (z 2^lead), the last bits of which do not matter, as it is the same for all tokens, and
    // 2^44 / z with what the fast exponential lacks.
    static __device__ void prepare(Shared *s, u64 z) {
        const int lead = lead_of(z);
        const double r = 9223372036854775808.0 / static_cast<double>(z << lead);
        s->inverse = r >= 0.9999999999999999 ? ~0ull : static_cast<u64>(r * 18446744073709551616.0);
        const double share = ldexp(r, lead - 19) * (1.0 + 5.1e-8);
        s->share_hi = static_cast<float>(share);
        s->share_lo = static_cast<float>(share - s->share_hi);
    }
    __device__ __forceinline__ RestSum(const Weights<T> &a, const Kept &b, const float *draft_probs, int tokens, u64 z, const Shared *s)
        : w(a), kept(b), q(draft_probs), vocab(tokens), shift(20 - lead_of(z)), inverse(s->inverse), share_hi(s->share_hi), share_lo(s->share_lo) {}
    __device__ __forceinline__ u64 rest(u64 weight, int i) const {
        const u64 mine = __umul64hi(weight << 19, inverse) >> shift;
        const unsigned bits = __float_as_uint(fminf(fmaxf(q[i], 0.f), 1.f));
        const int up = static_cast<int>(bits >> 23) - 88;  // 2^62 of a 24-bit significand
        const u64 s = (bits & 0x7fffffu) | 0x800000u, theirs = up >= 0 ? s << up : up > -24 ? s >> -up : 0;
        return mine > theirs ? mine - theirs : 0;
    }
    __device__ __forceinline__ float light_rest(float weight, float share) const {  // weight: as light_weights gives it
        return fmaxf(__fmaf_rn(weight, share_hi, weight * share_lo) - fmaxf(share, 0.f), 0.f);
    }
    __device__ __forceinline__ void add(float l, int i) {
        if (!kept.order(l, i)) return;
        float p, e;
        w.exponent(l, &p, &e);
        if (w.heavy(p)) h += rest(w.heavy_weight(p, e), i);
        else c += light_rest(w.light_weight(p, e) * 0x1p-44f, q[i]);
    }
    __device__ __forceinline__ u64 sum() const { return h + to_whole(c * 0x1p62f); }
    __device__ __forceinline__ static u64 up(float x) {
        const u64 v = to_whole(x * 0x1p62f);
        return v + (static_cast<float>(v) < x * 0x1p62f ? 1 : 0);
    }
    // What token t of a vector adds to vector(), in h and c.
    __device__ __forceinline__ void token(const uint4 *at, int first, int t) {
        if (Type<T>::largest(Type<T>::larger(at[0], at[1])) < kept.value) return;
        const float share = first + t >= 0 && first + t < vocab ? q[first + t] : 0.f;
        const unsigned special = light_weights(w, kept, at, [&](int u, u64 two) {
            float a, b;
            split_f32(two, &a, &b);
            if (u == t >> 1) c = light_rest(t & 1 ? b : a, share);
        });
        if (special >> t & 1) add(Type<T>::one(at, t), first + t);
    }
    __device__ __forceinline__ u64 vector(const uint4 *at, int first) {
        constexpr int P = Type<T>::kPer;
        if (Type<T>::largest(Type<T>::larger(at[0], at[1])) < kept.value) return 0;
        alignas(16) float share[P];
        if (first >= 0 && first + P <= vocab && (reinterpret_cast<uintptr_t>(q + first) & 15) == 0) {
#pragma unroll
            for (int u = 0; u < P; u += 4) *reinterpret_cast<float4 *>(&share[u]) = *reinterpret_cast<const float4 *>(q + first + u);
        } else {
#pragma unroll
            for (int u = 0; u < P; ++u) share[u] = first + u >= 0 && first + u < vocab ? q[first + u] : 0.f;
        }
        unsigned special = light_weights(w, kept, at, [&](int u, u64 two) {
            float a, b;
            split_f32(two, &a, &b);
            c += light_rest(a, share[2 * u]) + light_rest(b, share[2 * u + 1]);
        });
        for (; special; special &= special - 1) {
            const int u = __ffs(special) - 1;
            add(Type<T>::one(at, u), first + u);
        }
        return sum();
    }
};

// A row's slice in this block, and the cluster around it.
template <typename T>
struct Row {
    static constexpr int kPer = Type<T>::kPer;
    Shared *s;
    const uint4 *data;
    int warp, lane, block, blocks;
    int vectors, rounds, first;  // vectors of the slice, of a thread; index of the first vector's first element (which may lie before the slice)
    int parity, histogram;

    __device__ __forceinline__ void spread(int v, float *x) const {
        Type<T>::spread(data[2 * v], x);
        Type<T>::spread(data[2 * v + 1], x + Type<T>::kVector);
    }
    // Warp w takes a stretch of neighbouring vectors, so that index order is the order of warps, rounds, lanes and elements.
    __device__ __forceinline__ int vector(int round) const { return (warp * rounds + round) * 32 + lane; }

    template <typename F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll 1
        for (int k = 0; k < rounds; ++k) {
            const int v = vector(k);
            if (v >= vectors) break;
            float x[kPer];
            spread(v, x);
#pragma unroll
            for (int u = 0; u < kPer; ++u) f(x[u], first + v * kPer + u);
        }
    }
    // The first warp's values to every block; its lanes then read one of each.  What they make of them it tells the others: a warp less to issue
    // the same for.
    template <int N = 1>
    __device__ __forceinline__ void exchange(u64 a, u64 b = 0, u64 c = 0) {
        parity ^= 1;
        if (static_cast<int>(threadIdx.x) < blocks) {
            st_block_u64(at_block(&s->slot[parity][0][block], threadIdx.x), a);
            if (N > 1) st_block_u64(at_block(&s->slot[parity][1][block], threadIdx.x), b);
            if (N > 2) st_block_u64(at_block(&s->slot[parity][2][block], threadIdx.x), c);
        }
        cluster_barrier();
    }
    __device__ __forceinline__ u64 exchanged(int value) const { return lane < blocks ? s->slot[parity][value][lane] : 0; }
    __device__ __forceinline__ void say(u64 a, u64 b = 0, u64 c = 0) {
        if (lane == 0) {
            s->said[parity][0] = a;
            s->said[parity][1] = b;
            s->said[parity][2] = c;
        }
    }
    // The blocks' values (the first warp's): their sum, and that over the blocks before this one; `more`: something else for this block to hear.
    __device__ __forceinline__ u64 exchange_sum(u64 mine, u64 *before, u64 more = 0) {
        exchange(mine);
        if (warp == 0) {
            const u64 v = exchanged(0), upto = warp_prefix(v, lane), b = __shfl_sync(0xffffffffu, upto - v, block);
            say(__shfl_sync(0xffffffffu, upto, 31), b, more);
        }
        __syncthreads();
        *before = s->said[parity][1];
        return s->said[parity][0];
    }
    // The warps' sums to by_warp.
    __device__ __forceinline__ void warp_sums(u64 n, u64 *by_warp) {
        n = warp_sum(n);
        if (lane == 0) by_warp[warp] = n;
    }
    // Their sum, in the first warp.
    __device__ __forceinline__ u64 block_sum(const u64 *by_warp) const { return warp == 0 ? warp_sum(lane < kWarps ? by_warp[lane] : 0) : 0; }
    // The sum of `make()` over this block's slice, which leaves those over the warps' stretches in s->warp, over the blocks before it, and over all.
    struct Total {
        u64 mine, before, all;
    };
    template <typename M>
    __device__ __forceinline__ Total total(M make) {
        u64 n = 0;
#pragma unroll 1
        for (int k = 0; k < rounds; ++k) n += vector_sum(make, vector(k));
        __syncthreads();
        warp_sums(n, s->warp);
        __syncthreads();
        const u64 mine = block_sum(s->warp);
        Total t;
        t.all = exchange_sum(mine, &t.before, mine);
        t.mine = s->said[parity][2];
        return t;
    }
    template <typename M>
    __device__ __forceinline__ u64 vector_sum(M make, int v) const {
        auto a = make();
        return v < vectors ? a.vector(data + 2 * v, first + v * kPer) : 0;
    }
    // The first token at which the sum over the slice, taken just before by total() or tally(), exceeds `target` (less than it): its index, in
    // s->found. Called by the whole block. The stretch of the warp that it falls to is looked at by all warps, a round each.
    //
    // Sums are whole numbers from vectors on, so within a vector, whose tokens may each be less than one, they are taken as they are: exact sums and
    // 32-bit ones, of the very terms that the vector's sum has. So where that is not 0, neither is each of them, and what is found weighs something:
    // never a token that is masked, dropped or not the slice's.
    template <typename M>
    __device__ __forceinline__ void find(M make, u64 target) {
        u64 before, upto;
        const int w = first_past(s->warp, 0, target, &before), v = warp < rounds ? (w * rounds + warp) * 32 + lane : vectors;
        const u64 mine = vector_sum(make, v), all = warp_sum(mine);
        __syncthreads();
        if (lane == 0) s->scan[1][warp] = all;
        __syncthreads();
        int j = first_past(s->scan[1], before, target, &upto);
        // tally() adds tokens one by one, which may be a rounding more than this: then the last one of the stretch that weighs anything. There is one, as each
        // token of a nucleus weighs two units at least: with those behind it, fewer than 2^19 and none heavier, it weighs more than 1 - top_p >= 2^-24
        // of 2^44 units.
        const bool short_of = upto + s->scan[1][j] <= target;
        if (short_of) j = 31 - __clz(__ballot_sync(0xffffffffu, lane < kWarps && s->scan[1][lane % kWarps] > 0) | 1u);
        if (warp != j) return;
        const u64 prefix = upto + warp_prefix(mine, lane);
        const unsigned past = __ballot_sync(0xffffffffu, prefix > target), some = __ballot_sync(0xffffffffu, mine > 0);
        const int owner = past && !short_of ? __ffs(past) - 1 : 31 - __clz(some | 1u);
        upto = __shfl_sync(0xffffffffu, prefix - mine, owner);
        const int at = min(__shfl_sync(0xffffffffu, v, owner), vectors - 1);  // a vector of the slice, whatever the sums are
        auto a = make();
        if (lane < kPer) a.token(data + 2 * at, first + at * kPer, lane);
        const u64 h = upto + warp_prefix(a.h, lane);
        const float c = warp_prefix(static_cast<float>(a.c), lane);
        const unsigned any = __ballot_sync(0xffffffffu, a.h > 0 || a.c > 0.f);
        const unsigned here = any & __ballot_sync(0xffffffffu, h > target || a.up(c) > target - h);
        if (lane == 0) s->found = first + at * kPer + (here && !short_of ? __ffs(here) - 1 : 31 - __clz(any | 1u));
    }

    // The first of kWarps numbers at which their sum, with `before`, exceeds `target` (the last one if none does), and the sum before it.
    __device__ __forceinline__ int first_past(const u64 *n, u64 before, u64 target, u64 *sum_before) const {
        const u64 v = lane < kWarps ? n[lane] : 0, upto = before + warp_prefix(v, lane);
        const unsigned past = __ballot_sync(0xffffffffu, upto > target && lane < kWarps) | 1u << (kWarps - 1);
        const int at = __ffs(past) - 1;
        *sum_before = __shfl_sync(0xffffffffu, upto - v, at);
        return at;
    }
    // Inclusive sums over the block's threads.
    template <typename N>
    __device__ __forceinline__ N block_prefix(N v) {
        N *scan = reinterpret_cast<N *>(s->scan[0]);
        const N upto = warp_prefix(v, lane);
        __syncthreads();
        if (lane == 31) scan[warp] = upto;
        __syncthreads();
        const N w = lane < kWarps ? scan[lane] : 0;
        return upto + __shfl_sync(0xffffffffu, warp_prefix(w, lane) - w, warp);
    }

    // A histogram over the cluster's tokens (bin(l, i) < 0: not counted) and the first bin at which the number (MASS: weight) of tokens from
    // bin 0 on reaches `target`; kBins if none does.  What comes before it and lies in it is left in shared memory.
    template <bool MASS, typename B>
    __device__ __forceinline__ int reach(const Weights<T> &w, u64 target, bool near_end, B bin) {
        new_histogram();
        over(near_end, [&](float l, int i) {
            const int b = bin(l, i);
            if (b < 0) return;
            atomicAdd(&s->count[histogram][b], 1u);
            if (MASS) {
                const u64 v = w.weight(l);
                const unsigned low = static_cast<unsigned>(v), was = atomicAdd(&s->mass[histogram][b][0], low);
                const unsigned high = static_cast<unsigned>(v >> 32) + (was + low < low ? 1 : 0);
                if (high) atomicAdd(&s->mass[histogram][b][1], high);
            }
        });
        return reached<MASS>(target);
    }
    __device__ __forceinline__ void new_histogram() {
        histogram ^= 1;
        s->count[histogram][threadIdx.x] = 0;
        s->mass[histogram][threadIdx.x][0] = s->mass[histogram][threadIdx.x][1] = 0;
        __syncthreads();
    }
    // Each token of the slice, or of those near a nucleus' end.
    template <typename F>
    __device__ __forceinline__ void over(bool near_end, F f) const {
        if (near_end) {
            for (int i = threadIdx.x; i < static_cast<int>(s->nears); i += kThreads)
                f(value_of(s->near_end[i]), static_cast<int>(0xffffffffu - static_cast<unsigned>(s->near_end[i])));
        } else {
            each(f);
        }
    }
    // The blocks' histograms, which are all complete, added up: this thread's bin's number and weight. A block adds up its share of the bins and
    // tells the others: with each reading all of the others' 16 x 6 KB that took 10,000 cycles.
    template <bool MASS>
    __device__ __forceinline__ void merge(u64 *n, u64 *m) {
        const int share = kBins / blocks, bin = threadIdx.x % share, other = threadIdx.x / share;
        *m = 0;
        if (blocks == 1) {
            *n = s->count[histogram][bin];
            if (MASS) *m = static_cast<u64>(s->mass[histogram][bin][1]) << 32 | s->mass[histogram][bin][0];
            return;
        }
        unsigned *counts = s->count[histogram ^ 1];  // free: all blocks have done with the last histogram
        const unsigned c = ld_block_u32(at_block(&s->count[histogram][block * share + bin], other));
        u64 w = 0;
        if (MASS) w = ld_block_u64(at_block(&s->mass[histogram][block * share + bin][0], other));
        counts[threadIdx.x] = c;
        if (MASS) s->list[threadIdx.x] = w;
        __syncthreads();
        unsigned count = 0;
        w = 0;
        for (int b = 0; b < blocks; ++b) {  // each thread for the block that it tells
            count += counts[b * share + bin];
            if (MASS) w += s->list[b * share + bin];
        }
        st_block_u32(at_block(&s->all_count[block * share + bin], other), count);
        if (MASS) st_block_u64(at_block(&s->all_mass[block * share + bin], other), w);
        cluster_barrier();
        *n = s->all_count[threadIdx.x];
        if (MASS) *m = s->all_mass[threadIdx.x];
    }
    template <bool MASS>
    __device__ __forceinline__ int reached(u64 target) {
        cluster_barrier();
        u64 n, m;
        merge<MASS>(&n, &m);
        if (threadIdx.x == 0) s->found = kBins;
        const u64 count = block_prefix(n), mass = MASS ? block_prefix(m) : 0;
        const u64 upto = MASS ? mass : count, in = MASS ? m : n;
        if (upto >= target && upto - in < target) {
            s->found = threadIdx.x;
            s->count_before = count - n;
            s->count_in = n;
            s->mass_before = mass - m;
        }
        __syncthreads();
        return s->found;
    }

    // The tokens for which `wanted` holds into the blocks' lists; how many there are in all.
    template <typename W>
    __device__ __forceinline__ int gather(W wanted, bool near_end = false) {
        if (threadIdx.x == 0) s->listed = 0;
        __syncthreads();
        over(near_end, [&](float l, int i) {
            if (!wanted(l, i)) return;
            const unsigned at = atomicAdd(&s->listed, 1u);
            if (at < kList) s->list[at] = static_cast<u64>(float_order_code(l)) << 32 | (0xffffffffu - static_cast<unsigned>(i));
        });
        __syncthreads();
        u64 before;
        return static_cast<int>(exchange_sum(s->listed, &before));
    }
    // The first block's threads get a token each of the n (at most kList) in all lists, in their order; 0 behind them.
    __device__ __forceinline__ u64 sorted_list(int n) {
        u64 key = 0;
        int at = threadIdx.x;
        for (int b = 0; b < blocks && at >= 0; ++b) {
            const int here = static_cast<int>(s->slot[parity][0][b]);  // from gather()'s exchange
            if (at < here) key = ld_block_u64(at_block(&s->list[at], b));
            at -= here;
        }
        return sort(key, n);
    }
    // Bitonic, descending, of the threads' keys, of which those from n on are 0.
    __device__ __forceinline__ u64 sort(u64 key, int n) {
        int side = 0;
        for (int k = 2; k < 2 * n; k *= 2)
            for (int j = k / 2; j > 0; j /= 2) {
                u64 other;
                if (j >= 32) {
                    s->sort[side][threadIdx.x] = key;
                    __syncthreads();
                    other = s->sort[side][threadIdx.x ^ j];
                    side ^= 1;
                } else {
                    other = __shfl_xor_sync(0xffffffffu, key, j);
                }
                const bool large = ((threadIdx.x & k) == 0) == ((threadIdx.x & j) == 0);
                key = large == (key > other) ? key : other;
            }
        __syncthreads();
        return key;
    }

    // Narrows `kept` to the tokens up to the one at which their number (MASS: weight) in descending order reaches `target`, which has `above` from
    // the tokens with l >= to. `from`: a logit below which none of them lies. False if what is left from there on does not reach it.
    // near_end: all tokens of from <= l < to are in the lists of those.
    template <bool MASS>
    __device__ __forceinline__ bool select(Kept *kept, const Weights<T> &w, u64 target, float from, float to = INFINITY, u64 above = 0, bool near_end = false) {
        const Kept prior = *kept;
        // bins of equal width first, which spread the logits best
        const float high = fminf(to, w.top), range = high - from, scale = range > 0.f && range < 3e38f ? kSpread / range : 0.f;
        auto linear = [&](float l, int i) {
            return l >= from && (l < to || to == INFINITY) && prior.order(l, i) ? min(static_cast<int>((high - l) * scale), kBins - 1) : -1;
        };
        const int bin = reach<MASS>(w, target - above, near_end, linear);
        if (bin == kBins) return false;
        above += MASS ? s->mass_before : s->count_before;
        if (s->count_in <= kList) {
            narrow<MASS>(kept, w, target, above, gather([&](float l, int i) { return linear(l, i) == bin; }, near_end));
            return true;
        }
        // then of equal numbers of codes, until a bin is one logit
        unsigned c0, c1;
        {
            unsigned least = 0xffffffffu, most = 0;
            over(near_end, [&](float l, int i) {
                if (linear(l, i) != bin) return;
                least = min(least, float_order_code(l));
                most = max(most, float_order_code(l));
            });
            exchange_range(least, most, &c0, &c1);
        }
        for (;;) {
            const int bits = 32 - __clz(static_cast<int>(c1 - c0)), shift = max(bits - kBinBits, 0);
            const int b = reach<MASS>(w, target - above, near_end, [&](float l, int i) {
                const unsigned c = float_order_code(l);
                return prior.order(l, i) && c >= c0 && c <= c1 ? static_cast<int>((c1 - c) >> shift) : -1;
            });
            if (b == kBins) return false;  // not the case: the sums are whole numbers
            above += MASS ? s->mass_before : s->count_before;
            c1 -= static_cast<unsigned>(b) << shift;
            c0 = max(c0, c1 - ((1u << shift) - 1));
            if (shift == 0) break;
        }
        // all tokens of one logit: how many of them stay, and which one is the last
        const float value = value_of(static_cast<u64>(c1) << 32);
        u64 left = target - above;
        if (MASS) {
            const u64 each_one = w.weight(value);
            left = (left + each_one - 1) / each_one;
        }
        auto ties = [&] { return TieSum<T>(value, prior); };
        const Total n = total(ties);
        kept->value = value;
        kept->index = value == prior.value ? prior.index : 0x7fffffff;
        if (left >= n.all) return true;
        const bool here = left - 1 >= n.before && left - 1 < n.before + n.mine;
        if (here) find(ties, left - 1 - n.before);
        __syncthreads();
        u64 before;
        kept->index = static_cast<int>(exchange_sum(here ? s->found : 0, &before));
        return true;
    }
    // The same of the n tokens just gathered, which the target is reached among.
    template <bool MASS>
    __device__ __forceinline__ void narrow(Kept *kept, const Weights<T> &w, u64 target, u64 above, int n) {
        if (block == 0) {
            const u64 key = sorted_list(n);
            const u64 in = MASS ? (key ? w.weight(value_of(key)) : 0) : (key ? 1 : 0);
            const u64 upto = above + block_prefix(in);
            if (in && upto >= target && upto - in < target) s->last = key;
            __syncthreads();
            if (static_cast<int>(threadIdx.x) < blocks) st_block_u64(at_block(&s->last, threadIdx.x), s->last);
        }
        cluster_barrier();
        kept->value = value_of(s->last);
        kept->index = 0xffffffffu - static_cast<unsigned>(s->last);
    }

    // The kept tokens' sum z, and the nucleus of top_p of it. Returns the number of tokens listed, among which is the nucleus and all tokens
    // before its end, where they are few (LIST; at most n are kept); else narrows `kept` and returns 0.
    //
    // Where the nucleus ends is looked for with as few instructions a token as there are. The sum's pass counts tokens in a histogram of
    // eighths of powers of two: the heavier ones, and of the lighter ones an eighth (fp32: a quarter). That gives the place within some percent
    // or less; the next pass weighs what is before it and lists what is near it, exactly. (A histogram with weights of all tokens took 100
    // instructions and 3 atomics, of a cycle each, a token: 96 rows at temperature 1.6 took 326 us instead of then 180.)
    //
    // `kept_sum`, unless null: where the nucleus was narrowed down to by the lists, the total of what is kept (else left as it is).
    template <bool LIST>
    __device__ __forceinline__ int nucleus(Kept *kept, const Weights<T> &w, float top_p, int most, u64 *z, Total *kept_sum) {
        constexpr int kNoted = Type<T>::kVector;  // one of so many
        const Kept prior = *kept;
        if (threadIdx.x == 0) s->heavies = s->nears = 0;
        new_histogram();
        u64 n = 0, h = 0;
        const float counted_from = w.top - (static_cast<float>(kCounted) + 0.01f) / w.hi - 4.8e-7f * fabsf(w.top);
        {
            unsigned heavies = 0;
#pragma unroll 1
            for (int k = 0; k < rounds; ++k) {
                const int v = vector(k);
                if (v >= vectors) break;
                MassSum<T> m(w, prior);
                n += m.vector(data + 2 * v, first + v * kPer);
                h += m.h;
                heavies += m.h > 0 ? 1 : 0;
                auto note = [&](float l, bool every) {
                    const float y = (l - w.top) * w.hi;
                    const int bin = min(static_cast<int>(-static_cast<float>(kOctave) * y), kBins - 1);
                    if (y > -60.f && l > prior.value && (bin < kOctave * kCounted) == every) atomicAdd(&s->count[histogram][bin], 1u);
                };
                note(Type<T>::one(data + 2 * v, lane % kNoted), false);
                note(Type<T>::one(data + 2 * v + 1, lane % kNoted), false);
                if (Type<T>::largest(Type<T>::larger(data[2 * v], data[2 * v + 1])) >= counted_from) {
                    float x[kPer];
                    spread(v, x);
                    unsigned some = 0;
#pragma unroll
                    for (int u = 0; u < kPer; ++u)
                        if (x[u] >= counted_from) some |= 1u << u;
                    for (; some; some &= some - 1) note(Type<T>::one(data + 2 * v, __ffs(some) - 1), true);
                }
            }
            heavies = __reduce_add_sync(0xffffffffu, heavies);
            if (lane == 0 && heavies) atomicAdd(&s->heavies, heavies);
        }
        __syncthreads();
        warp_sums(n, s->warp);
        warp_sums(h, s->scan[1]);
        __syncthreads();
        n = block_sum(s->warp);
        h = block_sum(s->scan[1]);
        exchange<3>(n, h, s->heavies);
        if (warp == 0) {
            n = warp_sum(exchanged(0));
            h = warp_sum(exchanged(1));
            say(n, h, __reduce_add_sync(0xffffffffu, static_cast<unsigned>(exchanged(2))));
        }
        __syncthreads();
        *z = s->said[parity][0];
        h = s->said[parity][1];
        const unsigned heavies = static_cast<unsigned>(s->said[parity][2]);  // pieces with some
        u64 counted, none;
        merge<false>(&counted, &none);
        const u64 target = max(part_of(*z, top_p, true), 1ull);
        const float share = (1.f - top_p) * static_cast<float>(*z) * 0x1p-44f / static_cast<float>(most);
        // of at most `most` tokens, those lighter than an even share of what may be dropped are dropped all together
        const float lowest = share > 1e-30f ? fmaxf(w.top + (log2f(share) - 0.01f) / w.hi - 4.8e-7f * fabsf(w.top), kLowest) : kLowest;
        const bool in_heavy = target <= h;
        if (in_heavy && heavies <= kList) {
            const int listed = gather([&](float l, int i) { return (l >= w.top || w.heavy((l - w.top) * w.hi)) && prior.order(l, i); });
            if (listed <= kList && LIST) return listed;
            if (listed <= kList) {
                narrow<true>(kept, w, target, 0, listed);
                return 0;
            }
        }
        // The place by what was counted: the weight up to each bin's end, between the two nearest places whose weight is known, in proportion
        // to the counted one, and four times how far that may be off: a token's place in its bin, and how many stand for how many. (From the
        // lower place alone, 45% of wide nuclei of 152,064 tokens ended outside the lists and took one more pass.)
        const int bin = threadIdx.x;
        const bool every = bin < kOctave * kCounted;
        const float one = exp2f(-(static_cast<float>(bin) + 0.5f) / kOctave), c = (every ? 1 : kNoted) * static_cast<float>(counted);
        const float noted = block_prefix(c * one), number = block_prefix(c);
        const float square = block_prefix(c * one * one * (every ? 1e-3f : kNoted));
        const float goal = static_cast<float>(target) * 0x1p-44f;
        int low_bin = in_heavy ? -1 : kOctave * kHeavy - 1, high_bin = in_heavy ? kOctave * kHeavy - 1 : kBins - 1;
        float low = in_heavy ? 0.f : static_cast<float>(h) * 0x1p-44f, high = static_cast<float>(in_heavy ? h : *z) * 0x1p-44f;
        auto edge = [&](int b) { return w.top - static_cast<float>(b + 1) / (kOctave * w.hi); };
        for (int attempt = 0; attempt < 4 && w.simple; ++attempt) {
            __syncthreads();
            if (bin == 0) {
                s->to_bin = -1;
                s->from_bin = s->likely = s->least_from = kBins;
                s->at_to = 0.f;
                s->nears = 0;
                if (low_bin < 0) s->at_low[0] = s->at_low[1] = 0.f;
            }
            __syncthreads();
            if (bin == low_bin) {
                s->at_low[0] = noted;
                s->at_low[1] = square;
            }
            if (bin == high_bin) {
                s->at_high[0] = noted;
                s->at_high[1] = square;
            }
            __syncthreads();
            const float between = s->at_high[0] - s->at_low[0], part = between > 0.f ? (noted - s->at_low[0]) / between : 0.f;
            const float behind = s->at_high[1] - square, before = square - s->at_low[1];
            const float upto = low + part * (high - low);
            float off = 0.f;
            if (bin > low_bin && bin < high_bin)
                off = 4.f * sqrtf(fmaxf(before * (1.f - part) * (1.f - part) + behind * part * part, 0.f)) + 0.008f * fabsf(part * (1.f - part)) * between + 0.1f * one;
            if (upto + off < goal) atomicMax(&s->to_bin, bin);
            if (upto - off >= goal) atomicMin(&s->from_bin, bin);
            if (upto >= goal) atomicMin(&s->likely, bin);
            __syncthreads();
            int to_bin = s->to_bin, from_bin = s->from_bin;
            const int likely = min(s->likely, kBins - 1);
            if (bin == to_bin) s->at_to = number;
            if (bin == min(from_bin, kBins - 1)) s->at_from = number;
            if (bin == likely) s->at_likely = number - 0.5f * c;
            __syncthreads();
            const float most_near = 0.8f * kNear * blocks;
            if (s->at_from - s->at_to > most_near) {  // more than the lists hold: those nearest to where it most likely is
                if (bin < likely && number - c <= s->at_likely - 0.5f * most_near) atomicMax(&s->to_bin, bin);
                if (number >= s->at_likely + 0.5f * most_near) atomicMin(&s->least_from, bin);
                __syncthreads();
                to_bin = s->to_bin;
                from_bin = min(from_bin, max(s->least_from - 1, likely));
            }
            const float to = to_bin >= 0 ? edge(to_bin) : INFINITY, from = from_bin < kBins ? fmaxf(lowest, edge(from_bin)) : lowest;
            if (!(from < to && to > prior.value)) break;
            // what weighs before `to`, and a list of what lies from there to `from`
            const Kept upper{to, 0x7fffffff};
            n = 0;
#pragma unroll 1
            for (int k = 0; k < rounds; ++k) {
                const int v = vector(k);
                if (v >= vectors) break;
                const float largest = Type<T>::largest(Type<T>::larger(data[2 * v], data[2 * v + 1]));
                if (largest >= to) n += MassSum<T>(w, upper).vector(data + 2 * v, first + v * kPer);
                if (largest < from) continue;
                float x[kPer];
                spread(v, x);
                unsigned some = 0;
#pragma unroll
                for (int u = 0; u < kPer; ++u)
                    if (x[u] >= from && x[u] < to) some |= 1u << u;
                for (; some; some &= some - 1) {
                    const int i = first + v * kPer + __ffs(some) - 1;
                    const float l = Type<T>::one(data + 2 * v, __ffs(some) - 1);
                    if (!prior.order(l, i)) continue;
                    const unsigned at = atomicAdd(&s->nears, 1u);
                    if (at < kNear) s->near_end[at] = static_cast<u64>(float_order_code(l)) << 32 | (0xffffffffu - static_cast<unsigned>(i));
                }
            }
            __syncthreads();
            warp_sums(n, s->warp);
            __syncthreads();
            n = block_sum(s->warp);
            exchange<2>(n, s->nears);
            if (warp == 0) {
                n = warp_sum(exchanged(0));
                say(n, __reduce_max_sync(0xffffffffu, static_cast<unsigned>(exchanged(1))));
            }
            __syncthreads();
            const u64 above = s->said[parity][0], nears = s->said[parity][1];  // the most that a block has
            const u64 before_end = threadIdx.x < kWarps ? s->warp[threadIdx.x] : 0;
            if (nears <= kNear && above < target && select<true>(kept, w, target, from, to, above, true)) {
                if (kept_sum) *kept_sum = tally(*kept, w, before_end);
                return 0;
            }
            if (to_bin < 0) break;
            // not between these: once more, from a place whose weight is known now
            (above < target ? low_bin : high_bin) = to_bin;
            (above < target ? low : high) = static_cast<float>(above) * 0x1p-44f;
        }
        select<true>(kept, w, target, lowest);
        return 0;
    }
    // The total of what is kept: what weighs before the lists' tokens, by warps (the first threads' `before_end`), and the kept ones of those.
    __device__ __forceinline__ Total tally(const Kept &kept, const Weights<T> &w, u64 before_end) {
        unsigned(*sums)[2] = s->mass[histogram ^ 1];  // of the last histogram, which all blocks have done with
        __syncthreads();
        if (threadIdx.x < kWarps) sums[threadIdx.x][0] = sums[threadIdx.x][1] = 0;
        __syncthreads();
        over(true, [&](float l, int i) {
            if (!kept.order(l, i)) return;
            const int at = (i - first) / (kPer * 32 * rounds);
            const u64 v = w.weight(l);
            const unsigned low = static_cast<unsigned>(v), was = atomicAdd(&sums[at][0], low);
            const unsigned high = static_cast<unsigned>(v >> 32) + (was + low < low ? 1 : 0);
            if (high) atomicAdd(&sums[at][1], high);
        });
        __syncthreads();
        if (threadIdx.x < kWarps) s->warp[threadIdx.x] = before_end + (static_cast<u64>(sums[threadIdx.x][1]) << 32 | sums[threadIdx.x][0]);
        __syncthreads();
        const u64 mine = block_sum(s->warp);
        Total t;
        t.all = exchange_sum(mine, &t.before, mine);
        t.mine = s->said[parity][2];
        return t;
    }
    // Narrows `kept` to tokens of at least min_p. Weights never fall with the logits, so there is a largest one that is too small: each
    // warp looks for its code, in 31 places at a time.
    __device__ __forceinline__ void drop_below(Kept *kept, const Weights<T> &w, const Given &given) const {
        unsigned low = float_order_code(kLowest), high = float_order_code(w.top);  // the first may be too small, the last is not
        auto stays = [&](unsigned c) {
            float p, e;
            w.exponent(value_of(static_cast<u64>(c) << 32), &p, &e);
            return (p - given.floor_hi) + (e - given.floor_lo) >= 0.f;
        };
        if (stays(low)) return;
        while (high - low > 1) {
            const unsigned step = (high - low + 31) / 32, at = min(low + (lane + 1) * step, high);
            const int first = __ffs(__ballot_sync(0xffffffffu, at == high || stays(at))) - 1;
            high = __shfl_sync(0xffffffffu, at, first);
            low += first * step;
        }
        const float value = value_of(static_cast<u64>(low) << 32);
        if (value >= kept->value) *kept = {value, kNoIndex};  // also of the logit that another setting ended on, of which some are left
    }
    // The least and the largest of the cluster's codes.
    __device__ __forceinline__ void exchange_range(unsigned least, unsigned most, unsigned *c0, unsigned *c1) {
        const u64 mine = by_warp(least, most);
        exchange(warp == 0 ? join(mine) : 0);
        if (warp == 0) say(join(exchanged(0)));
        __syncthreads();
        const u64 all = s->said[parity][0];
        *c0 = 0xffffffffu - static_cast<unsigned>(all);
        *c1 = static_cast<unsigned>(all >> 32);
    }
    // The same of the threads' largest logits, and bounds from below for the 2 * blocks-th, 4 * blocks-th and 8 * blocks-th largest logit of all: what so
    // many of each block's warps have a logit of.
    __device__ __forceinline__ void exchange_largest(unsigned code, bool some, unsigned *least, unsigned *most, unsigned (&nth)[3]) {
        const u64 mine = by_warp(some ? code : 0xffffffffu, code);
        unsigned second = 0, fourth = 0, eighth = 0;
        u64 range = 0;
        if (warp == 0) {
            unsigned c = static_cast<unsigned>(mine >> 32);  // a warp's to a lane of 16: sorted, the largest first
#pragma unroll
            for (int k = 2; k <= kWarps; k *= 2)
#pragma unroll
                for (int j = k / 2; j > 0; j /= 2) {
                    const unsigned other = __shfl_xor_sync(0xffffffffu, c, j);
                    c = ((lane & k) == 0) == ((lane & j) == 0) ? max(c, other) : min(c, other);
                }
            second = __shfl_sync(0xffffffffu, c, 1);
            fourth = __shfl_sync(0xffffffffu, c, 3);
            eighth = __shfl_sync(0xffffffffu, c, 7);
            range = join(mine);
        }
        exchange<3>(range, static_cast<u64>(second) << 32 | fourth, eighth);
        if (warp == 0) {
            const u64 none = ~0ull, b = lane < blocks ? exchanged(1) : none, d = lane < blocks ? exchanged(2) : none;
            second = __reduce_min_sync(0xffffffffu, static_cast<unsigned>(b >> 32));
            fourth = __reduce_min_sync(0xffffffffu, static_cast<unsigned>(b));
            eighth = __reduce_min_sync(0xffffffffu, static_cast<unsigned>(d));
            say(join(exchanged(0)), static_cast<u64>(second) << 32 | fourth, eighth);
        }
        __syncthreads();
        const u64 all = s->said[parity][0];
        *least = 0xffffffffu - static_cast<unsigned>(all);
        *most = static_cast<unsigned>(all >> 32);
        nth[0] = static_cast<unsigned>(s->said[parity][1] >> 32);
        nth[1] = static_cast<unsigned>(s->said[parity][1]);
        nth[2] = static_cast<unsigned>(s->said[parity][2]);
    }
    // A warp's largest and (turned round) least code to each of kWarps lanes.
    __device__ __forceinline__ u64 by_warp(unsigned least, unsigned most) {
        least = __reduce_min_sync(0xffffffffu, least);
        most = __reduce_max_sync(0xffffffffu, most);
        __syncthreads();
        if (lane == 0) s->scan[0][warp] = static_cast<u64>(most) << 32 | (0xffffffffu - least);
        __syncthreads();
        return lane < kWarps ? s->scan[0][lane] : 0;
    }
    __device__ __forceinline__ static u64 join(u64 v) {
        return static_cast<u64>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(v >> 32))) << 32 |
               __reduce_max_sync(0xffffffffu, static_cast<unsigned>(v));
    }

    // The token of the weights `make()`, of which `t` is the total taken just before, at u of their sum.
    template <typename M>
    __device__ __forceinline__ void pick(M make, const Total &t, float u, long long *id) {
        const u64 target = place_of(u, t.all);
        if (target < t.before || target >= t.before + t.mine) return;
        find(make, target - t.before);
        __syncthreads();
        if (threadIdx.x == 0) *id = s->found;
    }
};

// log2 of a number in (0, 1] in two parts: the logarithm in 32 bits, and what is missing from 2^hi to the number.
__device__ __forceinline__ void log2_of(float x, const uint2 *table, float *hi, float *lo) {
    *hi = fmaxf(fminf(log2f(x), 0.f), -140.f);
    int shift;
    const unsigned s = Weights<float>::significand(*hi, 0.f, table, &shift);
    const float scaled = ldexpf(x, 28 + shift);  // exact
    *lo = (scaled - static_cast<float>(s & ~127u) - static_cast<float>(s & 127u)) / static_cast<float>(s) * 1.4426950409f;
}

// What row r is drawn by, into this block's shared memory.  One warp.
template <typename T, bool VERIFY>
__device__ __forceinline__ void give(const Draw &g, long long r, size_t row_at, Shared *s, int lane) {
    int setting = static_cast<int>(r), draft = -1;
    if (VERIFY) {  // the first sequence whose rows r is among
        setting = g.n_seqs;
        // their first rows ascend: 32 places at a time, until 32 sequences are left (each 32 sequences in turn: 80 us more for 2048 of 3 drafts
        // of 4000 tokens, which take 224)
        int q0 = 0;
        for (int q1 = g.n_seqs; q1 - q0 > 32;) {
            const int step = (q1 - q0 + 31) / 32, at = min(q0 + lane * step, q1 - 1);
            const unsigned upto = __ballot_sync(0xffffffffu, g.cu_drafts[at] + static_cast<long long>(at) <= r);
            q0 = min(q0 + max(31 - __clz(upto), 0) * step, q1 - 1);
            q1 = min(q0 + step, q1);
        }
        const int q = q0 + lane;
        int a = 0, b = -1;
        if (q < g.n_seqs) a = g.cu_drafts[q], b = g.cu_drafts[q + 1];
        const bool here = q < g.n_seqs && a >= 0 && b >= a && b <= g.n_drafts && r >= a + q && r <= b + q;
        const unsigned found = __ballot_sync(0xffffffffu, here);
        if (found) {
            setting = q0 + __ffs(found) - 1;
            draft = __shfl_sync(0xffffffffu, r < b + q ? static_cast<int>(r) - q : -1, __ffs(found) - 1);
        }
    }
    if (lane == 0) {
        Given v{};
        v.token = v.draft = -1;
        if (!VERIFY || setting < g.n_seqs) {
            v.u = g.uniforms[VERIFY ? 2 * r + 1 : r];
            const float temperature = g.temperature ? g.temperature[setting] : g.temperature_all;
            const float min_p = g.min_p ? g.min_p[setting] : g.min_p_all;
            const float top_p = g.top_p ? g.top_p[setting] : g.top_p_all;
            v.top_k = g.top_k ? g.top_k[setting] : g.top_k_all;
            if (VERIFY && draft >= 0) {
                const long long x = g.drafts[draft];
                if (x >= 0 && x < g.vocab) {
                    v.draft = draft;
                    v.token = static_cast<int>(x);
                    v.logit = Type<T>::one(g.logits, row_at + x);
                    v.accept = fminf(fmaxf(g.uniforms[2 * r], 0.f), 0x1.fffffep-1f);  // NaN: 0
                    v.share = g.draft_probs ? fmaxf(g.draft_probs[static_cast<size_t>(draft) * g.draft_probs_stride + x], 0.f) : 1.f;
                }
            }
            v.state = temperature > 0.f ? kDrawn : kGreedy;
            v.hi = 1.f;
            if (v.state == kDrawn) {
                // log2(e) / T by one step of a division in two parts. Within these temperatures neither part leaves the range of 32 bits; beyond
                // them a weight is one or nothing.
                const float d = fminf(fmaxf(temperature, 1e-30f), 1e30f);
                v.hi = 1.4426950216f / d;
                v.lo = (__fmaf_rn(-v.hi, d, 1.4426950216f) + 1.9259629e-8f) / d;
            }
            v.least = -200.f / v.hi;
            v.floor_hi = -INFINITY;
            if (v.state == kDrawn && min_p > 0.f) {
                v.floor_hi = g.floor_hi_all;
                v.floor_lo = g.floor_lo_all;
                if (g.min_p) log2_of(fminf(min_p, 1.f), s->table, &v.floor_hi, &v.floor_lo);
            }
            v.top_p = v.state == kGreedy || !(top_p < 1.f) ? 1.f : fmaxf(top_p, 0.f);
            if (v.top_k < 0 || v.top_k >= g.vocab) v.top_k = 0;
            if (v.state == kGreedy) v.top_k = 1;
        }
        s->given = v;
    }
    __syncwarp();
}

// Whether the draft is accepted, of s->drafted and the sum s->z; if not, what its rest is taken by.  Called by all threads.
template <typename T>
__device__ __forceinline__ bool judge(const Given &given, Shared *s) {
    if (threadIdx.x == 0) {
        const bool yes = static_cast<double>(given.accept) * static_cast<double>(given.share) * static_cast<double>(s->z) <
                         static_cast<double>(s->drafted);
        s->found = yes;
        if (!yes) RestSum<T>::prepare(s, s->z);
    }
    __syncthreads();
    return s->found;
}

// WHOLE: no row has a setting that drops tokens. What that needs fits 40 registers, so three blocks share an SM instead of two.
template <typename T, bool VERIFY, bool WHOLE>
__global__ void __launch_bounds__(kThreads, WHOLE ? 3 : 2) draw_kernel(const __grid_constant__ Draw g) {
    extern __shared__ __align__(16) unsigned char smem[];
    Row<T> row;
    Shared *s = row.s = reinterpret_cast<Shared *>(smem);
    row.data = reinterpret_cast<const uint4 *>(smem + shared_bytes(WHOLE));
    {
        unsigned r, n;
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
        row.block = r;
        row.blocks = n;
    }
    row.warp = threadIdx.x >> 5;
    row.lane = threadIdx.x & 31;
    row.parity = row.histogram = 0;
    const long long r = blockIdx.x / row.blocks;
    if (threadIdx.x < 64) s->table[threadIdx.x] = g.table[threadIdx.x];
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    pdl_launch_dependents();
    pdl_wait();  // no global-memory access before this point
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all blocks run: their shared memory may be written to

    const size_t row_at = static_cast<size_t>(r) * g.logits_stride;
    constexpr int P = Row<T>::kPer, V = Type<T>::kVector, kBatch = WHOLE ? 4 : 8;
    const int begin = min(row.block * g.slice, g.vocab), n = min(g.slice, g.vocab - begin);
    const T *from = static_cast<const T *>(g.logits) + row_at + begin;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(from) & 15) / static_cast<int>(sizeof(T));
    row.first = begin - off;
    row.vectors = n > 0 ? (off + n + P - 1) / P : 0;
    row.rounds = (row.vectors + kThreads - 1) / kThreads;
    const uint4 *whole = reinterpret_cast<const uint4 *>(from - off);
    const int full0 = off ? 1 : 0, full1 = (off + n) / V, loads = 2 * row.vectors;
    uint4 v[kBatch];
    auto request = [&](int k0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int at = (k0 + j) * kThreads + threadIdx.x;
            v[j] = make_uint4(Type<T>::kMasked, Type<T>::kMasked, Type<T>::kMasked, Type<T>::kMasked);
            if (at >= full0 && at < full1) v[j] = ldg_nc_v4(whole + at);
        }
    };
    request(0);
    if (row.block == 0 && row.warp == 0) {
        give<T, VERIFY>(g, r, row_at, s, row.lane);
        const unsigned *from_here = reinterpret_cast<const unsigned *>(&s->given);
        constexpr int kWords = static_cast<int>(sizeof(Given) / 4);
        for (int i = row.lane; i < (row.blocks - 1) * kWords; i += 32)
            st_block_u32(at_block(from_here + i % kWords, i / kWords + 1), from_here[i % kWords]);
    }
    // ---- the slice into shared memory, and the largest logit ----
    uint4 most = make_uint4(Type<T>::kMasked, Type<T>::kMasked, Type<T>::kMasked, Type<T>::kMasked);
    for (int k0 = 0; k0 * kThreads < loads; k0 += kBatch) {
        if (k0 > 0) request(k0);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int at = (k0 + j) * kThreads + threadIdx.x;
            if (at >= loads) break;
            if (at < full0 || at >= full1) {  // the slice's ends: element by element
                alignas(16) T part[V];
                *reinterpret_cast<uint4 *>(part) = v[j];
                for (int e = 0; e < V; ++e)
                    if (at * V + e >= off && at * V + e < off + n) part[e] = from[at * V + e - off];
                v[j] = *reinterpret_cast<uint4 *>(part);
            }
            const_cast<uint4 *>(row.data)[at] = v[j];
            most = Type<T>::larger(most, v[j]);
        }
    }
    const float mine = Type<T>::largest(most);  // this thread's
    unsigned least, largest, nth[3];
    if (WHOLE) row.exchange_range(0u, float_order_code(mine), &least, &largest);
    else row.exchange_largest(float_order_code(mine), mine > -INFINITY, &least, &largest, nth);
    const float top = value_of(static_cast<u64>(largest) << 32);

    // ---- what is left of the row ----
    const Given &given = s->given;  // here since the exchange
    if (given.state == kNotDrawn) return;  // a row behind the sequences: left as it is
    long long *id = g.ids + r;
    const bool probs = !VERIFY && g.probs;
    float *probs_to = probs ? g.probs + r * g.probs_stride : nullptr;
    const int end = begin + max(n, 0);
    if (top == -INFINITY) {
        if (row.block == 0 && threadIdx.x == 0) *id = -1;
        if (probs)
            for (int i = begin + threadIdx.x; i < end; i += kThreads) probs_to[i] = 0.f;
        return;
    }
    const Weights<T> weights(top, given, s->table);
    Kept kept{-INFINITY, kNoIndex};
    auto mass = [&] { return MassSum<T>(weights, kept); };
    const int top_k = WHOLE ? 0 : given.top_k;
    const bool by_p = !WHOLE && given.top_p < 1.f, by_floor = !WHOLE && given.floor_hi > -INFINITY;
    u64 z = 0;
    float cut = kLowest;  // a logit below which none of the kept tokens lies
    if (by_floor && !(top_k > 0 && by_p)) cut = fmaxf(cut, top + (given.floor_hi - 0.01f) / weights.hi - 4.8e-7f * fabsf(top));
    typename Row<T>::Total sums{};
    bool finish = false;
    int candidates = 0;
    auto list_all = [&] {
        candidates = row.gather([&](float l, int) { return l >= cut; });
        finish = candidates <= kList;
    };
    auto drop_light = [&] { return max(part_of(z, given.top_p, true), 1ull); };  // what the nucleus has to weigh, of the sum z
    if (top_k > 0) {
        // A bound from below: what each block has enough of, or the top_k-th largest of the threads' maxima.
        bool bounded = g.vocab <= kList;
        unsigned code = 0;
        if (top_k == 1) code = largest;
        else if (top_k <= 128)
            for (int j = 2; j >= 0; --j)
                if (top_k <= (2 << j) * row.blocks && (2 << j) * row.blocks <= 128) code = nth[j];
        if (code > float_order_code(-INFINITY)) {
            cut = fmaxf(cut, value_of(static_cast<u64>(code) << 32));
            bounded = true;
        } else if (top < 3.4e38f) {
            row.new_histogram();
            const float range = top - value_of(static_cast<u64>(least) << 32), scale = range > 0.f && range < 3e38f ? kSpread / range : 0.f;
            if (mine > -INFINITY) atomicAdd(&s->count[row.histogram][min(static_cast<int>((top - mine) * scale), kBins - 1)], 1u);
            const int bin = row.template reached<false>(top_k);
            if (bin < kBins) {
                cut = fmaxf(cut, top - (static_cast<float>(bin) + 1.001f) * (range / kSpread) - 4.8e-7f * fabsf(top));
                bounded = true;
            }
        }
        if (bounded) list_all();
    } else if (by_p) {
        candidates = row.template nucleus<true>(&kept, weights, given.top_p, g.vocab, &z, by_floor ? nullptr : &sums);
        finish = candidates > 0;
    } else if (by_floor) {
        list_all();
    }
    if (finish) {
        // ---- few tokens: the first block goes on with them alone ----
        if (row.block == 0) {
            const u64 key = row.sorted_list(candidates);
            if (!probs) cluster_barrier();  // the others leave
            const int i = 0xffffffffu - static_cast<unsigned>(key), rank = threadIdx.x;
            const float l = value_of(key);
            bool stays = key != 0 && (top_k == 0 || rank < top_k);
            float p, e;
            weights.exponent(l, &p, &e);
            u64 w = stays ? weights.weight(l) : 0;
            if (by_p) {
                const u64 upto = row.block_prefix(w);
                __syncthreads();
                if (threadIdx.x == kThreads - 1) s->z = upto;
                __syncthreads();
                if (top_k > 0) z = s->z;  // else that of all tokens
                stays = stays && upto - w < drop_light();
            }
            stays = stays && (p - given.floor_hi) + (e - given.floor_lo) >= 0.f;
            if (!stays) w = 0;
            // the kept ones come first: their number, and their sum
            const int left = __syncthreads_count(stays);
            if (VERIFY || probs) {
                const u64 upto = row.block_prefix(w);
                if (threadIdx.x == kThreads - 1) s->z = upto;
                if (VERIFY && threadIdx.x == 0) s->drafted = 0;
                if (rank == left - 1) s->last = key;
                __syncthreads();
            }
            if (probs) {
                if (static_cast<int>(threadIdx.x) < row.blocks && threadIdx.x > 0) {
                    st_block_u64(at_block(&s->last, threadIdx.x), s->last);
                    st_block_u64(at_block(&s->z, threadIdx.x), s->z);
                }
                cluster_barrier();
            }
            u64 weight = w;
            if (VERIFY && given.token >= 0) {
                if (stays && i == given.token) s->drafted = w;
                __syncthreads();
                if (judge<T>(given, s)) {
                    if (threadIdx.x == 0) *id = kAccepted;
                    return;
                }
                u64 over = stays && i != given.token ? w : 0;
                if (g.draft_probs) {
                    const RestSum<T> rest(weights, kept, g.draft_probs + static_cast<size_t>(given.draft) * g.draft_probs_stride, g.vocab, s->z, s);
                    over = stays ? rest.rest(w, i) >> 18 : 0;  // in 2^-44
                }
                if (__syncthreads_or(over != 0)) weight = over;
            }
            // in index order, with the weights of 45 bits behind the indices
            const u64 by_index = row.sort(stays ? static_cast<u64>(kMaxVocab - 1 - i) << 45 | weight : 0, left);
            weight = by_index & ((1ull << 45) - 1);
            const u64 upto = row.block_prefix(weight);
            if (threadIdx.x == kThreads - 1) s->z = upto;
            __syncthreads();
            const u64 target = place_of(given.u, s->z);
            if (upto > target && upto - weight <= target) *id = kMaxVocab - 1 - static_cast<int>(by_index >> 45);
        } else {
            cluster_barrier();
        }
        if (!probs) return;
        kept.value = value_of(s->last);
        kept.index = 0xffffffffu - static_cast<unsigned>(s->last);
        z = s->z;
    }
    if (!finish) {
        if (top_k > 0) {
            row.template select<false>(&kept, weights, top_k, cut);
            if (by_p) row.template nucleus<false>(&kept, weights, given.top_p, top_k, &z, by_floor ? nullptr : &sums);
        }
        if (by_floor) row.drop_below(&kept, weights, given);
        if (sums.all == 0) sums = row.total(mass);
        z = sums.all;
    }

    // ---- the distribution ----
    if (probs) {
        const float scale = 1.f / static_cast<float>(z);
        const bool wide = (reinterpret_cast<uintptr_t>(probs_to + row.first) & 15) == 0;
#pragma unroll 1
        for (int k = 0; k < row.rounds; ++k) {
            const int at = row.vector(k), i0 = row.first + at * P;
            if (at >= row.vectors) break;
            float y[P];
#pragma unroll
            for (int e = 0; e < P; ++e) y[e] = 0.f;
            unsigned special = light_weights(weights, kept, row.data + 2 * at, [&](int u, u64 two) {
                split_f32(mul_f32x2(two, pair_f32(0x1p44f * scale, 0x1p44f * scale)), &y[2 * u], &y[2 * u + 1]);
            });
            if (wide && i0 >= begin && i0 + P <= end) {
#pragma unroll
                for (int e = 0; e < P; e += 4) __stcs(reinterpret_cast<float4 *>(probs_to + i0 + e), make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]));
            } else {
#pragma unroll
                for (int e = 0; e < P; ++e)
                    if (i0 + e >= begin && i0 + e < end) probs_to[i0 + e] = y[e];
            }
            for (; special; special &= special - 1) {
                const int e = __ffs(special) - 1;
                const float l = Type<T>::one(row.data + 2 * at, e);
                if (!kept.order(l, i0 + e) || i0 + e < begin || i0 + e >= end) continue;
                float p, rest;
                weights.exponent(l, &p, &rest);
                probs_to[i0 + e] = (weights.heavy(p) ? static_cast<float>(weights.heavy_weight(p, rest)) : weights.light_weight(p, rest)) * scale;
            }
        }
        if (finish) return;
    }

    // ---- the token ----
    if (VERIFY && given.token >= 0) {
        if (threadIdx.x == 0) {
            s->drafted = kept.order(given.logit, given.token) ? weights.weight(given.logit) : 0;
            s->z = z;
        }
        if (judge<T>(given, s)) {
            if (row.block == 0 && threadIdx.x == 0) *id = kAccepted;
            return;
        }
        if (g.draft_probs) {
            const float *q = g.draft_probs + static_cast<size_t>(given.draft) * g.draft_probs_stride;
            auto rest = [&] { return RestSum<T>(weights, kept, q, g.vocab, z, s); };
            const typename Row<T>::Total t = row.total(rest);
            if (t.all > 0) {
                row.pick(rest, t, given.u, id);
                return;
            }
        } else {
            auto others = [&] { return MassSum<T, true>(weights, kept, given.token); };
            const typename Row<T>::Total t = row.total(others);
            if (t.all > 0) {
                row.pick(others, t, given.u, id);
                return;
            }
        }
        sums = row.total(mass);  // the warps' sums are wanted again
    }
    row.pick(mass, sums, given.u, id);
}

// Each sequence's accepted drafts, the token drawn at its first row that did not accept, and -1 behind it.  A warp to a sequence.
__global__ void __launch_bounds__(128) settle_kernel(const Draw g) {
    const int q = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    if (q >= g.n_seqs) return;
    const int a = g.cu_drafts[q], b = g.cu_drafts[q + 1];
    if (a < 0 || b < a || b > g.n_drafts) return;
    long long *ids = g.ids + a + q;
    const int n = b - a;
    int taken = n;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const unsigned no = __ballot_sync(0xffffffffu, i0 + lane < n && ids[i0 + lane] != kAccepted);
        if (no) {
            taken = i0 + __ffs(no) - 1;
            break;
        }
    }
    for (int i = lane; i <= n; i += 32)
        if (i != taken) ids[i] = i < taken ? g.drafts[a + i] : -1;
    if (lane == 0) g.accepted[q] = taken;
}

template <typename... Args>
cudaError_t launch_cluster(void (*kernel)(Args...), int grid, int cluster, int threads, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, bool VERIFY, bool WHOLE>
dspark_status launch(Draw g, int sms, cudaStream_t stream) {
    auto *kernel = draw_kernel<T, VERIFY, WHOLE>;
    static std::atomic<unsigned long long> configured{0};  // a bit a device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev >= 64 || !(configured.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(shared_bytes(WHOLE)) + kMostSlice + 128);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(sample)");
        if (dev < 64) configured.fetch_or(1ull << dev);
    }
    // Blocks of a row's cluster: a block takes some time whatever its slice, about that of 8 KB of it, and two of them (three, where nothing is
    // dropped) share an SM. 96 rows of 151936 (bf16, nuclei) over 4 | 8 | 16 blocks 198 | 121 | 207 us, 28 of them (fp32) over 8 | 16 44 | 61. An
    // estimate: it counts SMs, where a cluster has to fit into one of the GPU's groups of them, and tries powers of two alone.
    constexpr int kShare = WHOLE ? 3 : 2;
    constexpr long long kGoodSlice = 227 * 1024 / kShare - 1024 - static_cast<long long>(shared_bytes(WHOLE)) - 64;
    const long long size = sizeof(T), bytes = g.vocab * size, slots = static_cast<long long>(kShare) * sms;
    int blocks = 0;
    long long least = 0;
    for (int b = 1; b <= kMaxBlocks; b *= 2) {
        const long long slice = (bytes + b - 1) / b, cost = (g.rows * static_cast<long long>(b) + slots - 1) / slots * (slice + 8 * 1024);
        if (slice <= (b < kMaxBlocks ? kGoodSlice : kMostSlice) && (blocks == 0 || cost < least)) {
            blocks = b;
            least = cost;
        }
    }
    const int per = 16 / static_cast<int>(size);  // whole vectors: all slices begin at the same place of one
    g.slice = ((g.vocab + blocks - 1) / blocks + per - 1) / per * per;
    const size_t smem = shared_bytes(WHOLE) + g.slice * size + 64;  // what stands before the slice's first vector and fills its last one
    e = launch_cluster(kernel, g.rows * blocks, blocks, kThreads, smem, stream, g);
    return e == cudaSuccess ? DSPARK_OK : cuda_fail(e, VERIFY ? "verify_drafts" : "sample");
}

dspark_status check(const char *who, const void *logits, int dtype, int rows, int vocab, long long stride, const dspark_filters &f) {
    if (rows < 0 || vocab < 1) return fail(DSPARK_ERR_INVALID, "%s: bad sizes rows=%d vocab=%d", who, rows, vocab);
    if (vocab > kMaxVocab) return fail(DSPARK_ERR_UNSUPPORTED, "%s: vocab %d > %d", who, vocab, kMaxVocab);
    if (rows > 0x7fffffff / kMaxBlocks) return fail(DSPARK_ERR_UNSUPPORTED, "%s: %d rows", who, rows);
    if (dtype < DSPARK_FP16 || dtype > DSPARK_FP32) return fail(DSPARK_ERR_INVALID, "%s: unknown type %d", who, dtype);
    if (rows > 1 && stride < 0) return fail(DSPARK_ERR_INVALID, "%s: negative row stride", who);
    if (!f.temperature && !(f.temperature_all >= 0.f))
        return fail(DSPARK_ERR_INVALID, "%s: temperature %g is negative or not a number", who, f.temperature_all);
    if (!f.top_p && !(f.top_p_all >= 0.f && f.top_p_all <= 1.f)) return fail(DSPARK_ERR_INVALID, "%s: top_p %g is not in 0..1", who, f.top_p_all);
    if (!f.min_p && !(f.min_p_all >= 0.f && f.min_p_all <= 1.f)) return fail(DSPARK_ERR_INVALID, "%s: min_p %g is not in 0..1", who, f.min_p_all);
    if (!f.top_k && f.top_k_all < 0) return fail(DSPARK_ERR_INVALID, "%s: top_k %d is negative", who, f.top_k_all);
    if (!aligned(f.temperature, 4) || !aligned(f.top_p, 4) || !aligned(f.min_p, 4) || !aligned(f.top_k, 4) ||
        !aligned(logits, dtype == DSPARK_FP32 ? 4 : 2))
        return fail(DSPARK_ERR_INVALID, "%s: misaligned pointer", who);
    return DSPARK_OK;
}

struct Table {
    uint2 entry[64];
    Table() {
        for (int j = 0; j < 64; ++j) {
            const double x = std::exp2(28.0 + j / 64.0);
            const float as_float = static_cast<float>(x);
            entry[j].x = static_cast<unsigned>(std::llrint(x));
            std::memcpy(&entry[j].y, &as_float, 4);
        }
    }
};

template <bool VERIFY>
dspark_status run(Draw g, int dtype, const dspark_filters &f, cudaStream_t stream) {
    g.temperature = f.temperature;
    g.top_p = f.top_p;
    g.min_p = f.min_p;
    g.top_k = f.top_k;
    g.temperature_all = f.temperature_all;
    g.top_p_all = f.top_p_all;
    g.min_p_all = f.min_p_all;
    g.top_k_all = f.top_k_all;
    if (!f.min_p && f.min_p_all > 0.f) {
        const double least = std::log2(static_cast<double>(f.min_p_all));
        g.floor_hi_all = static_cast<float>(least);
        g.floor_lo_all = static_cast<float>(least - g.floor_hi_all);
    }
    static const Table table;
    std::memcpy(g.table, table.entry, sizeof g.table);
    int sms = 0;
    const dspark_status st = static_cast<dspark_status>(current_sm_count(&sms));
    if (st != DSPARK_OK) return st;
    const bool whole = !f.temperature && f.temperature_all > 0.f && !f.top_k && (f.top_k_all == 0 || f.top_k_all >= g.vocab) && !f.top_p &&
                       f.top_p_all >= 1.f && !f.min_p && f.min_p_all <= 0.f;
    auto *go = dtype == DSPARK_FP32   ? (whole ? launch<float, VERIFY, true> : launch<float, VERIFY, false>)
               : dtype == DSPARK_BF16 ? (whole ? launch<__nv_bfloat16, VERIFY, true> : launch<__nv_bfloat16, VERIFY, false>)
                                      : (whole ? launch<__half, VERIFY, true> : launch<__half, VERIFY, false>);
    return go(g, sms, stream);
}

}  // namespace

}  // namespace dspark

extern "C" dspark_status dspark_sample(const dspark_sample_args *a, dspark_stream_t stream) {
    using namespace dspark;
    const char *who = "sample";
    if (!a) return fail(DSPARK_ERR_INVALID, "%s: null arguments", who);
    const dspark_status st = check(who, a->logits, a->dtype, a->rows, a->vocab, a->logits_stride, a->filters);
    if (st != DSPARK_OK || a->rows == 0) return st;
    if (!a->logits || !a->uniforms || !a->ids) return fail(DSPARK_ERR_INVALID, "%s: null pointer argument", who);
    if (!aligned(a->uniforms, 4) || !aligned(a->ids, 8) || !aligned(a->probs, 4))
        return fail(DSPARK_ERR_INVALID, "%s: misaligned pointer", who);
    if (a->probs && a->rows > 1 && a->probs_stride < a->vocab)
        return fail(DSPARK_ERR_INVALID, "%s: rows of probs overlap (stride %lld, vocab %d)", who, a->probs_stride, a->vocab);
    Draw g{};
    g.logits = a->logits;
    g.uniforms = a->uniforms;
    g.ids = reinterpret_cast<long long *>(a->ids);
    g.probs = a->probs;
    g.logits_stride = a->logits_stride;
    g.probs_stride = a->probs_stride;
    g.rows = a->rows;
    g.vocab = a->vocab;
    return run<false>(g, a->dtype, a->filters, stream);
}

extern "C" dspark_status dspark_verify_drafts(const dspark_verify_args *a, dspark_stream_t stream) {
    using namespace dspark;
    const char *who = "verify_drafts";
    if (!a) return fail(DSPARK_ERR_INVALID, "%s: null arguments", who);
    if (a->n_seqs < 0 || a->n_drafts < 0) return fail(DSPARK_ERR_INVALID, "%s: bad sizes n_seqs=%d n_drafts=%d", who, a->n_seqs, a->n_drafts);
    if (a->n_drafts > 0x7fffffff - a->n_seqs) return fail(DSPARK_ERR_UNSUPPORTED, "%s: %d drafts", who, a->n_drafts);
    const int rows = a->n_drafts + a->n_seqs;
    const dspark_status st = check(who, a->logits, a->dtype, rows, a->vocab, a->logits_stride, a->filters);
    if (st != DSPARK_OK || a->n_seqs == 0) return st;
    if (!a->logits || !a->uniforms || !a->ids || !a->accepted || !a->cu_drafts || (a->n_drafts > 0 && !a->drafts))
        return fail(DSPARK_ERR_INVALID, "%s: null pointer argument", who);
    if (!aligned(a->uniforms, 4) || !aligned(a->ids, 8) || !aligned(a->drafts, 8) || !aligned(a->accepted, 4) || !aligned(a->cu_drafts, 4) ||
        !aligned(a->draft_probs, 4))
        return fail(DSPARK_ERR_INVALID, "%s: misaligned pointer", who);
    if (a->draft_probs && a->n_drafts > 1 && a->draft_probs_stride < 0) return fail(DSPARK_ERR_INVALID, "%s: negative row stride", who);
    Draw g{};
    g.logits = a->logits;
    g.uniforms = a->uniforms;
    g.cu_drafts = a->cu_drafts;
    g.drafts = reinterpret_cast<const long long *>(a->drafts);
    g.draft_probs = a->draft_probs;
    g.ids = reinterpret_cast<long long *>(a->ids);
    g.accepted = a->accepted;
    g.logits_stride = a->logits_stride;
    g.draft_probs_stride = a->draft_probs_stride;
    g.rows = rows;
    g.vocab = a->vocab;
    g.n_seqs = a->n_seqs;
    g.n_drafts = a->n_drafts;
    dspark_status done = run<true>(g, a->dtype, a->filters, stream);
    if (done != DSPARK_OK) return done;
    const cudaError_t e = launch_pdl(settle_kernel, dim3((g.n_seqs + 3) / 4), dim3(128), 0, stream, g);
    return e == cudaSuccess ? DSPARK_OK : cuda_fail(e, "verify_drafts (settle)");
}
