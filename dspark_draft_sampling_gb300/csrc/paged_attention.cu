// Attention of a chunk of new tokens over the paged cache, on tcgen05 tensor cores.
//
// Rows.  The query heads that share a kv head, of consecutive tokens, are the rows of one 128-row query
// tile: row r is head r % group of token r / group.  So a decode step of a few heads, a draft block and a long
// prompt chunk are the same kernel: S = Q K^T is a 128 x 128 tile of rows against 128 keys, and O += P V follows
// with P = exp2(scale' S - m) in 16 bits, read from tensor memory.  Tensor memory holds two such pipelines
// ("streams", 128 columns of S and up to 128 of O each), so that one stream's products run while the other's softmax
// does.  With long chunks (PAIR) the streams are two query tiles over the same keys; with at most 128 rows they are the
// even and odd key tiles of one query tile, joined at the end.
//
// Softmax.  A thread owns a row.  The running maximum only moves (and O is only rescaled) when a tile's maximum
// exceeds it by more than 8 powers of two (fp16: 4), and sums stay exact enough in 32 bits, as the final division takes the
// common factor out.  P is rounded to the inputs' type for the second product, which rounds each weight
// once (unit roundoff 2^-11 or 2^-8, of the size of the output's own rounding); its sum is taken in 32 bits before
// that rounding.  An fp16 weight below 2^-14 keeps fewer bits and one below 2^-25 none, which many keys would feel: at the maximum
// 66,000 of 2^-25 are 0.2 % of it.  So fp16's P is 2^7 times as large, at most 2^11 with 5 powers of two to spare for
// roundings of very large scores: what a weight loses is 2^-32 of the maximum, and a million keys' 2^-12.
//
// Work.  All (sequence, kv head, query tile) items, each with its own number of 128-key tiles, form one
// sequence of tiles that the thread blocks, one to an SM, take in equal contiguous ranges, or, where cutting would cost more
// than it gains, an item each.  Every block finds its range from the lengths on the device, so nothing about them has
// to be known on the host.  An item cut by a range's end
// leaves partial sums (32-bit O, maximum, sum) in the workspace; the block that arrives last joins them in
// block order, many of them in two steps, so the result does not depend on which one that is.
//
// Measured (GB300). 8192 tokens after 8192, 32 / 8 heads of 128: 0.93 ms, 1.77 PFLOP/s, for ten launches after a pause;
// 1.02 ms, 1.62 PFLOP/s, under the power cap, where the library's matrix product sustains 1.75. 1-8 tokens over 16,000-66,000
// keys: 182 us for 1.2 GB, 98 % of a copy's rate. 16 x 7 tokens over 300-6000 keys: 42 us for 183 MB, of which about 30 are that
// stream, the rest start and joins. Chunks of 90-1500 tokens in a window of 1000, 28 / 4 heads of 64: 69 us, where the chain
// of one stream (scores, softmax, second product) takes 2500 cycles a pair of key tiles and the products 1024. One token
// over 777 keys: 11 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kv_cache.cuh"
#include "tc.cuh"

namespace dspark {

namespace {

constexpr int kTile = 128;                    // query rows of a tile, keys of a tile
constexpr int kThreads = 384;                 // warps 0-3, 4-7: softmax of stream 0, 1; 8: copies; 9: MMA issue; 10, 11: none
// Registers of a softmax and of another thread: the launch gives all kThreads 168, and 256 * 208 + 128 * 80 is less.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80, kLaunchRegs = 168;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "more registers than the block was launched with");
constexpr int kTmemCols = 512;
constexpr size_t kSmemData = 224 * 1024;      // query tiles and the ring of key and value tiles
constexpr size_t kSmemBytes = 227 * 1024;
// An item's fixed cost, in key tiles. With 1, 2, 3, 4, 6: 16 blocks of 7 tokens over 300-6000 keys (pages in two copies then) 44.7,
// 44.8, 46.0, 46.0, 49.4 us; chunks in a window of 1000 70.7, 68.8, 69.0, 68.2, 69.4; 4 chunks of 64 tokens over 3000 keys 36.8, 34.9, 32.7, 33.0, 33.5.
constexpr int kItemCost = 2;
// Powers of two by which a row's maximum may lag. With 0, 4, 8: prompt of 8192 tokens after 8192 1176, 1023, 1019 us (bf16).
template <bool BF16>
constexpr float kRescale = BF16 ? 8.f : 4.f;
// Powers of two that P is larger by; a row's sum is, too.
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;
// Rows (rounded up to a power of two) x parts of an item from which its parts are joined in two steps. One step | two: 49 tokens over
// 8720 keys in 35 parts 52 | 32 us, 64 tokens over 8000 keys in 19 parts 47 | 39; 32 tokens over 1000 keys in 10 parts 21.4 | 22.6.
constexpr int kTwoSteps = 2048;
static_assert(kMaxCtas < 256, "arrivals are counted in bytes");

struct Attention {
    void *out;
    float *lse;
    long long out_token, out_head;
    const int *rows, *cu_new;
    int tokens, group, n_seqs, layer, causal, window, chunk_tiles;  // chunk_tiles: query tiles of the longest chunk (hint)
    int tile_tokens;    // tokens of a 128-row tile
    unsigned cut;       // what cutting items costs, in key tiles
    float scale;
    float *partials;
    unsigned *arrivals;
    unsigned long long timeout_ns, stall_ns;  // of waits at the block's end, of the debug entry's
    uint32_t tries;                            // of the pipeline's waits
};

template <int D, bool PAIR>
struct Shape {
    static constexpr int QT = PAIR ? 2 : 1;
    static constexpr int kHalves = D / 64;                       // 64-element column blocks of 128 bytes
    static constexpr uint32_t kTileBytes = kTile * D * 2;
    static constexpr int kStages = static_cast<int>((kSmemData - QT * kTileBytes) / kTileBytes);
    static constexpr size_t kSlotFloats = size_t(kTile) * (D + 4);  // partial of one query tile: O, maximum, sum; maximum, sum of a joined O
};

size_t slot_bytes(int head_dim) { return 4 * size_t(kTile) * (head_dim + 4); }

struct Seq {
    int row, n, length, q0;  // table row, new tokens, tokens, first query token
};

__device__ __forceinline__ Seq load_seq(const CacheView &c, const Attention &g, int s) {
    Seq q;
    const int a = min(max(g.cu_new[s], 0), g.tokens), b = min(g.cu_new[s + 1], g.tokens);
    q.q0 = a;
    q.n = max(b - a, 0);
    q.row = g.rows ? g.rows[s] : s;
    q.length = 0;
    const int most = c.max_pages << c.page_shift;  // below 2^30
    bool bad = static_cast<unsigned>(q.row) >= static_cast<unsigned>(c.max_seqs);
    if (bad) {
        q.row = 0;
    } else {
        const int length = c.length[q.row];
        q.length = min(max(length, 0), most);
        bad = q.length != length;
    }
    if (bad && q.n > 0) atomicOr(c.status, kStatusIndex);
    return q;
}

// Keys [begin, end) that some token of query tile i (of `step` tokens) of a sequence sees, and the key tiles [lo, hi) they lie in.
struct Keys {
    int begin, end, lo, hi;
};

__device__ __forceinline__ Keys keys_of(const Attention &g, const Seq &q, int i, int step) {
    const int off = q.length - q.n, first = i * step, last = min(first + step, q.n) - 1;
    Keys k;
    k.end = g.causal ? min(q.length, max(off + last + 1, 0)) : q.length;
    k.begin = g.window > 0 ? max(0, off + first - g.window + 1) : 0;
    k.hi = (k.end + kTile - 1) / kTile;
    k.lo = k.begin < k.end ? k.begin / kTile : k.hi;
    return k;
}

// What an item counts among all tiles.
__device__ __forceinline__ int item_cost(const Attention &g, const Seq &q, int i, int step) {
    const Keys k = keys_of(g, q, i, step);
    return kItemCost + k.hi - k.lo;
}

// One stretch of an item that a block works on, as the copying warp hands it to the others.
struct Segment {
    int kv_head, tile;        // query tile of the sequence
    int lo, first, last;      // the item's first key tile; the stretch's, relative to it
    int tiles;                // of the whole item; -1: no more segments
    int begin, end;           // keys that some row of the item sees
    int q0, n, length;        // the sequence's first query token, its new tokens, its tokens
    int cf, cl;               // first and last block that work on the item (where that is more than one)
};

// Walks a block's range.
struct Walk {
    Seq q;
    int s, kv_head, i, n_tiles, step;
    unsigned per;              // key tiles of a block (the last one takes what is left, blocks behind it none)
    unsigned x, left, pos, at; // x: place within the item; pos: absolute place; at: the last segment's item's

    __device__ __forceinline__ bool next(const CacheView &c, const Attention &g, Segment *out) {
        while (left > 0) {
            if (i >= n_tiles) {
                i = 0;
                if (++kv_head == c.kv_heads) {
                    kv_head = 0;
                    do {
                        q = load_seq(c, g, ++s);
                    } while (q.n == 0);
                    n_tiles = (q.n + step - 1) / step;
                }
            }
            const Keys k = keys_of(g, q, i, step);
            const int tiles = k.hi - k.lo;
            const unsigned take = min(left, kItemCost + tiles - x);
            out->kv_head = kv_head;
            out->tile = i;
            out->lo = k.lo;
            out->begin = k.begin;
            out->end = k.end;
            out->tiles = tiles;
            out->first = max(static_cast<int>(x) - kItemCost, 0);
            out->last = max(static_cast<int>(x + take) - kItemCost, 0);
            out->q0 = q.q0;
            out->n = q.n;
            out->length = q.length;
            at = pos - x;
            const bool starts = x == 0;
            left -= take;
            pos += take;
            x = 0;
            ++i;
            if (out->last > out->first || (tiles == 0 && starts)) return true;
        }
        return false;
    }
};

__device__ __forceinline__ unsigned warp_scan(unsigned v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

__device__ __forceinline__ void tmem_ld_32(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Natural logarithm of a row's sum: sum / 2^kLift times 2^top.
template <bool BF16>
__device__ __forceinline__ float log_sum(float top, float sum) {
    constexpr float back = 1.f / static_cast<float>(1 << static_cast<int>(kLift<BF16>));
    return sum == 0.f ? -INFINITY : (top + lg2(sum * back)) * 0.6931471805599453f;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    uint32_t r;
    if (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ unsigned long long pair_u32(uint32_t a, uint32_t b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ unsigned long long pair_f32(float a, float b) { return pair_u32(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ void split_f32(unsigned long long v, float *a, float *b) {
    uint32_t x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(v));
    *a = __uint_as_float(x);
    *b = __uint_as_float(y);
}
__device__ __forceinline__ unsigned long long fma_f32x2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ unsigned long long add_f32x2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 32 lanes x 16 columns from registers; awaited with tmem_wait_st().
__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Lane l of four holds w[0..3] of its row; afterwards w[k] is the l-th of lane k's.
__device__ __forceinline__ void transpose_4(uint32_t (&w)[4][4], int lane) {
#pragma unroll
    for (int by = 1; by <= 2; by *= 2) {
        const bool upper = (lane & by) != 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j & by) continue;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? w[j][x] : w[j + by][x], by);
                if (upper) w[j][x] = got;
                else w[j + by][x] = got;
            }
        }
    }
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load_3d_plain(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// Key and value tiles lie in shared memory as [8-key group][64-element block][key of the group][64 elements], 128-byte rows
// with the 128-byte swizzle, so that one copy brings a page whatever its length and the groups are evenly spaced. With a copy for each
// block of a page ([block][key]) prompts over pages of 16 took a fifth longer: 8192 tokens after 8192 1117
// against 931 us, where the power cap does not hold it back.
template <int D>
__device__ __forceinline__ uint64_t smem_desc_tile(uint32_t addr, uint32_t leading) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(leading >> 4) << 16;
    d |= static_cast<uint64_t>((D * 16u) >> 4) << 32;  // from group to group
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
// Keys are the first product's B operand, K (head elements) contiguous; values the second's, N (head elements) contiguous, where the
// leading offset goes from one 64-element block to the next.
template <int D>
__device__ __forceinline__ uint64_t smem_desc_keys(uint32_t addr) { return smem_desc_tile<D>(addr, 16); }
template <int D>
__device__ __forceinline__ uint64_t smem_desc_values(uint32_t addr) { return smem_desc_tile<D>(addr, 1024); }

// What is joined at once: count parts of one item. A block that an item begins with keeps its part in its second slot, the
// others in their first, so the parts are a stride apart but for the first one, which may lie `lead` further on. Their maxima stand in
// column max_col of a part, their sums in the next.
struct Join {
    float *base;
    unsigned stride, lead;  // in floats
    int count, max_col;
    __device__ __forceinline__ float *part(int k) const { return base + (k * stride + (k == 0 ? lead : 0u)); }
};

// Joins columns c4, c4 + step, ... (of four values each) of one row: COLS columns of PARTS parts are in flight at a time. The
// result goes to the output, or, in 32 bits and not divided, in place of the first part.
template <bool BF16, int D, int COLS, int PARTS>
__device__ __forceinline__ void join_columns(const Join &j, int row, int c4, int step, float top, float inv, float sc, bool final,
                                             unsigned short *to) {
    float4 *joined = reinterpret_cast<float4 *>(j.part(0)) + row;
    for (; c4 < D / 4; c4 += COLS * step) {
        float4 acc[COLS];
#pragma unroll
        for (int q = 0; q < COLS; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < j.count; k0 += PARTS) {
            float w[PARTS];
            float4 o[PARTS][COLS];
#pragma unroll
            for (int u = 0; u < PARTS; ++u) {  // behind the last part: the last one again, with weight 0
                const float *p = j.part(min(k0 + u, j.count - 1));
                w[u] = k0 + u < j.count ? __ldcg(p + size_t(kTile) * j.max_col + row) : -INFINITY;
#pragma unroll
                for (int q = 0; q < COLS; ++q)
                    o[u][q] = __ldcg(reinterpret_cast<const float4 *>(p) + min(c4 + q * step, D / 4 - 1) * kTile + row);
            }
#pragma unroll
            for (int u = 0; u < PARTS; ++u) {
                const float k = w[u] == -INFINITY ? 0.f : ex2((w[u] - top) * sc);  // a part that saw nothing holds zeros
#pragma unroll
                for (int q = 0; q < COLS; ++q) {
                    acc[q].x += o[u][q].x * k;
                    acc[q].y += o[u][q].y * k;
                    acc[q].z += o[u][q].z * k;
                    acc[q].w += o[u][q].w * k;
                }
            }
        }
#pragma unroll
        for (int q = 0; q < COLS; ++q)
            if (c4 + q * step < D / 4) {
                if (final)
                    *reinterpret_cast<uint2 *>(to + (c4 + q * step) * 4) =
                        make_uint2(pack16<BF16>(acc[q].x * inv, acc[q].y * inv), pack16<BF16>(acc[q].z * inv, acc[q].w * inv));
                else
                    __stcg(joined + (c4 + q * step) * kTile, acc[q]);
            }
    }
}

constexpr int kSegments = 4;  // segments handed over ahead

// Barriers and small state behind the data area.
template <int STAGES>
struct Control {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_half[2], p_ready[2], o_full[2];
    uint64_t sync[2];   // softmax threads among themselves: per stream (PAIR), or [0] for both
    uint64_t seg_full[kSegments], seg_empty[kSegments];
    uint64_t drained, never;
    Segment segs[kSegments];
    uint32_t tmem, aborted;
    unsigned last[2];
    float max_sum[2][2][kTile];  // [stream][maximum, sum][row], one query tile's two streams
};

// As mbar_try_wait, suspended for up to `ns` nanoseconds.
__device__ __forceinline__ bool mbar_try_wait_for(uint64_t *bar, uint32_t parity, uint32_t ns) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(ns)
        : "memory");
    return ok != 0;
}

// A whole warp waits, `tries` times 1000 ns at most.  The lanes decide together at every turn, so that the warp stays converged:
// with each lane in a loop of its own the code behind the wait ran in pieces.  Turns are counted, as reading the clock takes longer than
// most waits and as this code stands in many places.
template <typename C>
__device__ __forceinline__ bool warp_wait(C *ctl, uint64_t *bar, uint32_t parity, const CacheView &c, uint32_t tries) {
#pragma unroll 1
    for (; !__all_sync(0xffffffffu, mbar_try_wait_for(bar, parity, 1000)); --tries) {
        if (tries == 0) {
            *static_cast<volatile uint32_t *>(&ctl->aborted) = 1;
            atomicOr(c.status, kStatusTimeout);
        }
        if (__any_sync(0xffffffffu, *static_cast<volatile uint32_t *>(&ctl->aborted))) return false;
    }
    return true;
}

// The next segment, read by one warp.
template <typename C>
__device__ __forceinline__ bool next_segment(C *ctl, uint32_t &n_seg, Segment *seg, const CacheView &c, uint32_t tries) {
    const uint32_t slot = n_seg % kSegments;
    if (!warp_wait(ctl, &ctl->seg_full[slot], (n_seg / kSegments) & 1, c, tries)) return false;
    ++n_seg;
    *seg = ctl->segs[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ctl->seg_empty[slot]);
    return seg->tiles >= 0;
}

template <bool BF16, int D, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv, const CacheView c,
                     const Attention g) {
    using S = Shape<D, PAIR>;
    using C = Control<S::kStages>;
    extern __shared__ __align__(1024) unsigned char smem[];  // swizzled tiles want 1024-byte alignment
    C *ctl = reinterpret_cast<C *>(smem + kSmemData);
    static_assert(sizeof(C) <= kSmemBytes - kSmemData, "control block does not fit");
    const uint32_t q_smem = smem_addr(smem), ring = q_smem + S::QT * S::kTileBytes;
    unsigned char *ring_ptr = smem + S::QT * S::kTileBytes;
    const int warp = (__shfl_sync(0xffffffffu, threadIdx.x >> 5, 0) + 8) % 12, lane = threadIdx.x & 31;
    const int step = g.tile_tokens * S::QT;  // tokens of an item

    if (warp == 8 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_q)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_kv)) : "memory");
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1);
        }
        mbar_init(&ctl->q_full, 1);
        mbar_init(&ctl->q_empty, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&ctl->s_full[s], 1);
            mbar_init(&ctl->p_half[s], 4);  // one arrival a warp
            mbar_init(&ctl->p_ready[s], 4);
            mbar_init(&ctl->o_full[s], 1);
            mbar_init(&ctl->sync[s], PAIR ? 128 : 256);
        }
        for (int i = 0; i < kSegments; ++i) {
            mbar_init(&ctl->seg_full[i], 1);
            mbar_init(&ctl->seg_empty[i], 9);  // the softmax warps and the MMA warp
        }
        mbar_init(&ctl->drained, 1);
        mbar_init(&ctl->never, 1);
        ctl->aborted = 0;
        fence_mbar_init();
    }
    if (warp == 9) tmem_alloc(&ctl->tmem, kTmemCols);
    pdl_launch_dependents();
    pdl_wait();  // no global-memory access before this point
    // Every sequence's cost.  Up to 32 sequences of few query tiles are left to the copying warp, a lane each.
    unsigned *cost = reinterpret_cast<unsigned *>(ring_ptr);  // the ring serves as scratch until the first copy
    const bool few = g.n_seqs <= 32 && g.chunk_tiles <= 4;
    if (!few) {
        const int of_seq = g.chunk_tiles <= 4 ? 1 : 32;  // threads to a sequence
        for (int s = threadIdx.x / of_seq; s < g.n_seqs; s += kThreads / of_seq) {
            const Seq q = load_seq(c, g, s);
            unsigned w = 0, most = 0;
            for (int i = threadIdx.x % of_seq; i * step < q.n; i += of_seq) {
                const unsigned v = item_cost(g, q, i, step);
                w += v;
                most = max(most, v);
            }
            if (of_seq == 32) {
                w = __reduce_add_sync(0xffffffffu, w);
                most = __reduce_max_sync(0xffffffffu, most);
            }
            if (threadIdx.x % of_seq == 0) {
                cost[s] = w;
                if (s < 32) cost[kMaxSeqs + s] = most, cost[kMaxSeqs + 32 + s] = (q.n + step - 1) / step;
            }
        }
        fence_proxy_async_smem();  // the scratch use comes before the copies into the ring
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8) {
            // ---- copies: query tiles, then keys and values of each tile through the ring; a lane to a page ----
            const int box = min(c.page_size, kTile), per_tile = kTile / box;
            uint32_t n_q = 0, n_seg = 0, put = 0;  // segments with keys, segments, ring entries so far
            Walk walk;
            walk.left = 0;
            walk.step = step;
            {
                // ---- this block's range of all items' tiles, and the item that it begins with ----
                // in 32 bits: the host has made sure that the tiles' number fits
                Seq mine{};
                unsigned w = 0, most = 0, items = 0;
                if (lane < g.n_seqs) {
                    if (few) {
                        mine = load_seq(c, g, lane);
                        for (; static_cast<int>(items) * step < mine.n; ++items) {
                            const unsigned v = item_cost(g, mine, items, step);
                            w += v;
                            most = max(most, v);
                        }
                    } else {
                        w = cost[lane];
                        most = cost[kMaxSeqs + lane];
                        items = cost[kMaxSeqs + 32 + lane];
                    }
                }
                unsigned total = w;
                for (int s = 32 + lane; s < g.n_seqs; s += 32) total += cost[s];
                total = __reduce_add_sync(0xffffffffu, total) * c.kv_heads;
                // not less than an item's fixed cost: 32 tokens over 1000 keys take 17 us, 21 in ranges of one tile; 7 over 2000 keys 12.0,
                // 14.2. Ranges of 4 and more pay for some (300 tokens 11.5 against 15.7), but one token over 776 keys takes 14.3 against 10.6.
                unsigned per = max((total + gridDim.x - 1) / gridDim.x, static_cast<unsigned>(kItemCost));
                // Where there are no more items than blocks and whole ones take little longer, a block takes an item: each then counts as
                // much as the longest. Single tiles are bound by memory, whose share of a block grows when others are done.
                most = __reduce_max_sync(0xffffffffu, most);
                const unsigned all = __reduce_add_sync(0xffffffffu, items) * c.kv_heads;
                const bool whole_items = g.n_seqs <= 32 && all <= gridDim.x && most <= per + (PAIR ? 0 : per / 4) + g.cut;
                if (whole_items) {
                    per = most;
                    w = items * most;
                    total = all * most;
                }
                walk.per = per;
                walk.pos = min(per * blockIdx.x, total);
                walk.left = min(per, total - walk.pos);
                if (walk.left > 0) {
                    unsigned before = 0;
                    for (int s0 = 0;; s0 += 32) {
                        if (s0 > 0) w = s0 + lane < g.n_seqs ? cost[s0 + lane] : 0;
                        const unsigned upto = before + warp_scan(w, lane) * c.kv_heads;
                        const unsigned past = __ballot_sync(0xffffffffu, upto > walk.pos);
                        if (past || s0 + 32 >= g.n_seqs) {  // the range lies within the sequences: found in the last stretch at the latest
                            const int l = past ? __ffs(past) - 1 : 0;
                            walk.s = s0 + l;
                            w = __shfl_sync(0xffffffffu, w, l);
                            before = __shfl_sync(0xffffffffu, upto, l) - w * c.kv_heads;
                            if (!few) mine = load_seq(c, g, s0 + lane < g.n_seqs ? s0 + lane : walk.s);
                            walk.q.row = __shfl_sync(0xffffffffu, mine.row, l);
                            walk.q.n = __shfl_sync(0xffffffffu, mine.n, l);
                            walk.q.length = __shfl_sync(0xffffffffu, mine.length, l);
                            walk.q.q0 = __shfl_sync(0xffffffffu, mine.q0, l);
                            break;
                        }
                        before = __shfl_sync(0xffffffffu, upto, 31);
                    }
                    walk.n_tiles = (walk.q.n + step - 1) / step;
                    walk.kv_head = (walk.pos - before) / w;
                    unsigned rem = walk.pos - before - walk.kv_head * w;
                    if (whole_items) {
                        walk.i = rem / per;
                        walk.x = 0;
                        walk.left = item_cost(g, walk.q, walk.i, step);
                    }
                    for (int i0 = 0; i0 < walk.n_tiles && !whole_items; i0 += 32) {
                        const unsigned v = i0 + lane < walk.n_tiles ? item_cost(g, walk.q, i0 + lane, step) : 0;
                        const unsigned upto = warp_scan(v, lane);
                        const unsigned past = __ballot_sync(0xffffffffu, upto > rem);
                        if (past) {
                            const int l = __ffs(past) - 1;
                            walk.i = i0 + l;
                            walk.x = rem - __shfl_sync(0xffffffffu, upto - v, l);
                            break;
                        }
                        rem -= __shfl_sync(0xffffffffu, upto, 31);
                    }
                }
            }
            bool ok = true;
            for (bool more = true; ok && more;) {
                Segment seg;
                more = walk.next(c, g, &seg);
                if (!more) seg.tiles = -1;
                seg.cf = seg.cl = blockIdx.x;
                if (more && (seg.first != 0 || seg.last != seg.tiles)) {
                    if (seg.first != 0) seg.cf = (walk.at + kItemCost) / walk.per;
                    if (seg.last != seg.tiles) seg.cl = (walk.at + kItemCost + seg.tiles - 1) / walk.per;
                }
                const uint32_t entry = n_seg % kSegments;
                if (n_seg >= kSegments && !(ok = warp_wait(ctl, &ctl->seg_empty[entry], ((n_seg / kSegments) & 1) ^ 1, c, g.tries))) break;
                ++n_seg;
                if (lane == 0) {
                    ctl->segs[entry] = seg;
                    mbar_arrive(&ctl->seg_full[entry]);
                }
                __syncwarp();
                if (!more || seg.tiles == 0) continue;
                if (n_q > 0 && !(ok = warp_wait(ctl, &ctl->q_empty, (n_q - 1) & 1, c, g.tries))) break;
                ++n_q;
                const int token = seg.q0 + seg.tile * step;
                if (lane == 0) {
                    const uint32_t rows_bytes = static_cast<uint32_t>(g.tile_tokens * g.group) * 128u;
                    mbar_arrive_expect_tx(&ctl->q_full, rows_bytes * S::kHalves * S::QT);
                    for (int t = 0; t < S::QT; ++t)
                        for (int h = 0; h < S::kHalves; ++h)
                            tma_load_3d_plain(q_smem + t * S::kTileBytes + h * (kTile * 128), &tm_q, h * 64, seg.kv_head * g.group,
                                              token + t * g.tile_tokens, &ctl->q_full);
                }
                const int *pages = c.table + static_cast<size_t>(walk.q.row) * c.max_pages;
                const int run = (g.layer * 2) * c.kv_heads + seg.kv_head, runs = c.layers * 2 * c.kv_heads, page_groups = c.page_size / 8;
                for (int t = seg.first; ok && t < seg.last; ++t) {
                    const int key = (seg.lo + t) * kTile + lane * box;  // first key of this lane's page
                    const bool mine = lane < per_tile && key < seg.end && key + box > seg.begin;  // pages that no row sees are not looked at
                    int page = 0;
                    if (mine) {
                        page = pages[key >> c.page_shift];
                        if (static_cast<unsigned>(page) >= static_cast<unsigned>(c.num_pages)) {
                            atomicOr(c.status, kStatusIndex);
                            page = c.num_pages;  // outside the tensor: reads as zeros
                        }
                    }
                    const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, mine));
                    const int group = (page * runs + run) * page_groups + (key & (c.page_size - 1)) / 8;  // a page may be longer than a tile
                    for (int w = 0; w < 2; ++w, ++put) {
                        const uint32_t st = put % S::kStages;
                        if (put >= S::kStages && !(ok = warp_wait(ctl, &ctl->empty[st], ((put / S::kStages) & 1) ^ 1, c, g.tries))) break;
                        if (lane == 0) mbar_arrive_expect_tx(&ctl->full[st], boxes * static_cast<uint32_t>(box) * D * 2);
                        __syncwarp();
                        if (mine)
                            tma_load_4d(ring + st * S::kTileBytes + lane * box * (D * 2), &tm_kv, 0, 0, 0, group + w * c.kv_heads * page_groups,
                                        &ctl->full[st]);
                    }
                }
            }
            // copies in flight land before the block ends, also after a wait that gave up
            for (uint32_t p = put > S::kStages ? put - S::kStages : 0; p < put; ++p)
                mbar_wait(&ctl->full[p % S::kStages], (p / S::kStages) & 1, g.timeout_ns);
            if (n_q) mbar_wait(&ctl->q_full, (n_q - 1) & 1, g.timeout_ns);
        } else if (warp == 9) {
            // ---- MMA issue: the warp runs as one, an elected lane issues ----
            constexpr uint32_t idesc_s = idesc_f16(BF16, kTile, kTile);
            constexpr uint32_t idesc_o = idesc_f16(BF16, kTile, D) | (1u << 16);  // B is N-contiguous
            uint32_t n_q = 0, n_seg = 0, base = 0;  // segments with keys, segments, key tiles before this segment
            uint32_t p_phase = 0;                   // one bit a stream: the phase of its next P
            bool ok = true;
            Segment seg;
            // Ring entries and their phases: key tile j of all is entry 2 * j, its values the next one.
            struct Entry {
                uint32_t st, phase;
            };
            auto entry = [&](uint32_t p) {
                const uint32_t turn = p / S::kStages;
                return Entry{__shfl_sync(0xffffffffu, p - turn * S::kStages, 0), turn & 1};
            };
            auto ready = [&](uint64_t *bar, uint32_t phase) { return warp_wait(ctl, bar, phase, c, g.tries); };
            auto issue_scores = [&](const int s, const Entry &e, bool frees_q) {
                const uint64_t a = smem_desc_sw128(q_smem + (PAIR ? s * S::kTileBytes : 0));
                const uint64_t b = smem_desc_keys<D>(ring + e.st * S::kTileBytes);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc_mma_f16(tmem + s * kTile, a + (((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4), b + (((k / 4) * 1024 + (k % 4) * 32) >> 4),
                               idesc_s, k != 0);
                tc_commit(&ctl->s_full[s]);
                if (!PAIR || s == 1) tc_commit(&ctl->empty[e.st]);
                if (frees_q) tc_commit(&ctl->q_empty);  // the segment's last scores free its query tiles
            };
            auto issue_values = [&](const int s, const Entry &e, const int half, bool add) {
                const uint64_t b = smem_desc_values<D>(ring + e.st * S::kTileBytes);
#pragma unroll
                for (int k = half * (kTile / 32); k < (half + 1) * (kTile / 32); ++k)
                    tc_mma_f16_ts(tmem + 2 * kTile + s * kTile, tmem + s * kTile + k * 8, b + ((k * D * 32) >> 4), idesc_o, add || k != 0);
            };
            // One step of stream s: its second product, then the scores of its next key tile.
            auto advance = [&](const int s, const Entry &v, const Entry &k, bool first, bool more, bool frees_q) {
                if (!ready(&ctl->p_half[s], (p_phase >> s) & 1)) return false;
                tc_fence_after();
                if (elect_one()) issue_values(s, v, 0, !first);
                __syncwarp();
                if (!ready(&ctl->p_ready[s], (p_phase >> s) & 1)) return false;
                p_phase ^= 1u << s;
                tc_fence_after();
                if (elect_one()) {
                    issue_values(s, v, 1, true);
                    if (!PAIR || s == 1) tc_commit(&ctl->empty[v.st]);
                    if (!more) tc_commit(&ctl->o_full[s]);
                    if (PAIR && more) issue_scores(s, k, frees_q);
                }
                __syncwarp();
                if (!PAIR && more) {
                    // these keys may be on their way still, and the values' slot was wanted back first
                    if (!ready(&ctl->full[k.st], k.phase)) return false;
                    tc_fence_after();
                    if (elect_one()) issue_scores(s, k, frees_q);
                    __syncwarp();
                }
                return true;
            };
            while (ok && next_segment(ctl, n_seg, &seg, c, g.tries)) {
                if (seg.tiles == 0) continue;
                const int nt = seg.last - seg.first;
                const int steps0 = PAIR ? nt : (nt + 1) / 2, steps1 = PAIR ? nt : nt / 2;
                const uint32_t p0 = 2 * base;
                base += nt;
                if (!(ok = ready(&ctl->q_full, n_q & 1))) break;
                ++n_q;
                {
                    const Entry k0 = entry(p0), k1 = PAIR ? k0 : entry(p0 + 2);
                    if (!(ok = ready(&ctl->full[k0.st], k0.phase))) break;
                    tc_fence_after();
                    if (elect_one()) issue_scores(0, k0, steps0 == 1 && steps1 == 0);
                    __syncwarp();
                    if (steps1 > 0) {
                        if (!PAIR && !(ok = ready(&ctl->full[k1.st], k1.phase))) break;
                        tc_fence_after();
                        if (elect_one()) issue_scores(1, k1, steps0 == 1);
                        __syncwarp();
                    }
                }
                for (int i = 0; i < steps0; ++i) {
                    if (PAIR) {
                        // both streams read the same tiles; the next keys have long arrived when they are looked at
                        const bool more = i + 1 < nt;
                        const Entry v = entry(p0 + 2 * i + 1), k = entry(p0 + 2 * i + 2);
                        if (!(ok = ready(&ctl->full[v.st], v.phase) && (!more || ready(&ctl->full[k.st], k.phase)))) break;
                        if (!(ok = advance(0, v, k, i == 0, more, false))) break;
                        if (!(ok = advance(1, v, k, i == 0, more, i + 2 == nt))) break;
                    } else {
                        const Entry v0 = entry(p0 + 4 * i + 1), k0 = entry(p0 + 4 * i + 4);
                        if (!(ok = ready(&ctl->full[v0.st], v0.phase))) break;
                        if (!(ok = advance(0, v0, k0, i == 0, i + 1 < steps0, i + 2 == steps0 && i + 1 >= steps1))) break;
                        if (i >= steps1) continue;
                        const Entry v1 = entry(p0 + 4 * i + 3), k1 = entry(p0 + 4 * i + 6);
                        if (!(ok = ready(&ctl->full[v1.st], v1.phase))) break;
                        if (!(ok = advance(1, v1, k1, i == 0, i + 1 < steps1, i + 2 == steps0))) break;
                    }
                }
            }
            if (elect_one()) tc_commit(&ctl->drained);
            __syncwarp();
            mbar_wait(&ctl->drained, 0, g.timeout_ns);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ---- softmax of stream s: a thread owns row r ----
        const int s = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + s * kTile + lanes, t_o = tmem + 2 * kTile + s * kTile + lanes;
        const float sc = g.scale * 1.4426950408889634f;
        const int row_token = r / g.group, row_head = r - row_token * g.group;
        uint32_t n_s = 0, n_seg = 0, n_o0 = 0, n_o1 = 0, n_sync = 0, base = 0;
        bool ok = true;
        if (g.stall_ns && !mbar_wait(&ctl->never, 0, g.stall_ns) && warp == 0 && lane == 0) atomicOr(c.status, kStatusTimeout);
        Segment seg;
        while (ok && next_segment(ctl, n_seg, &seg, c, g.tries)) {
            const int nt = seg.last - seg.first;
            const int token = seg.tile * step + (PAIR ? s * g.tile_tokens : 0) + row_token;  // of the chunk
            const bool real = row_token < g.tile_tokens && token < seg.n;
            const int pos = seg.length - seg.n + token;
            // keys that this row sees; rows that are none see all, as what they hold is not written
            const int see_hi = !real ? 0x7fffffff : g.causal ? min(seg.length, pos + 1) : seg.length;
            const int see_lo = real && g.window > 0 ? max(0, pos - g.window + 1) : 0;
            float m = -INFINITY, l = 0.f;
            const int steps = PAIR ? nt : (nt + 1 - s) / 2;
            const bool warp_real = __any_sync(0xffffffffu, real);
            for (int i = 0; i < steps && ok; ++i) {
                const int t = PAIR ? i : 2 * i + s;
                const int key0 = (seg.lo + seg.first + t) * kTile;
                if (!(ok = warp_wait(ctl, &ctl->s_full[s], n_s & 1, c, g.tries))) break;
                ++n_s;
                tc_fence_after();
                if (key0 < seg.begin || key0 + kTile > seg.end) {
                    // Values that no row of the item sees are whatever the pages hold, or were not copied: zeros, so that weights of 0
                    // stay 0.
                    const uint32_t p = 2 * (base + t) + 1, st = p % S::kStages;
                    if (!(ok = warp_wait(ctl, &ctl->full[st], (p / S::kStages) & 1, c, g.tries))) break;
                    const int first = max(seg.begin - key0, 0) * 8, last = min(seg.end - key0, kTile) * 8;
                    unsigned char *v = ring_ptr + st * S::kTileBytes;
                    for (int h = 0; h < S::kHalves; ++h) {
                        uint4 *at = reinterpret_cast<uint4 *>(v) + h * 64;
                        for (int b = r; b < first; b += kTile) at[b + (b & ~63) * (S::kHalves - 1)] = make_uint4(0u, 0u, 0u, 0u);
                        for (int b = last + r; b < kTile * 8; b += kTile) at[b + (b & ~63) * (S::kHalves - 1)] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                if (warp_real) {
                    uint32_t v[kTile];
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    const bool edge = __any_sync(0xffffffffu, key0 < see_lo || key0 + kTile > see_hi);
                    if (edge) {
                        // masked in place, a quarter at a time: few tiles have an edge, and their code stands here once
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            const int lo = see_lo - key0 - q * 32, hi = see_hi - key0 - q * 32;
                            if (!__any_sync(0xffffffffu, lo > 0 || hi < 32)) continue;
                            uint32_t w[32];
                            tmem_ld_32(t_s + q * 32, w);
                            tmem_wait_ld();
#pragma unroll
                            for (int u = 0; u < 32; ++u)
                                if (u < lo || u >= hi) w[u] = 0xff800000u;
                            tmem_st_32(t_s + q * 32, w);
                        }
                        tmem_wait_st();
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld_32(t_s + q * 32, v + q * 32);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < kTile; q += 8) {
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            top[w] = fmaxf(top[w], fmaxf(__uint_as_float(v[q + 2 * w]), __uint_as_float(v[q + 2 * w + 1])));
                    }
                    const float tile_max = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    const bool moves = real && (tile_max - m) * sc > kRescale<BF16>;  // also from -infinity
                    if (__any_sync(0xffffffffu, moves)) {
                        const float up = fmaxf(m, tile_max);
                        const float keep = m == -INFINITY ? 0.f : ex2((m - up) * sc);
                        if (i > 0) {
                            // the scores' arrival also says that this stream's earlier second products are done
#pragma unroll 1
                            for (int q = 0; q < D / 16; ++q) {
                                uint32_t o[16];
                                tmem_ld_16(t_o + q * 16, o);
#pragma unroll
                                for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * keep);
                                tmem_st_16(t_o + q * 16, o);
                            }
                        }
                        l *= keep;
                        m = up;
                    }
                    const float shift = m == -INFINITY ? 0.f : kLift<BF16> - m * sc;
                    const unsigned long long sc2 = pair_f32(sc, sc), shift2 = pair_f32(shift, shift);
                    unsigned long long sum2[2] = {0ull, 0ull};
                    // groups of 8 weights: one group's exponentials between the next one's arguments and the last one's sums,
                    // so that none of them waits for another's latency
                    unsigned long long x[kTile / 2];
                    uint32_t w[kTile / 2];
                    auto arguments = [&](int g8) {
#pragma unroll
                        for (int u = 4 * g8; u < 4 * g8 + 4; ++u) x[u] = fma_f32x2(pair_u32(v[2 * u], v[2 * u + 1]), sc2, shift2);
                    };
                    arguments(0);
                    arguments(1);
#pragma unroll
                    for (int g8 = 0; g8 <= kTile / 8; ++g8) {
                        if (g8 + 2 < kTile / 8) arguments(g8 + 2);
                        if (g8 < kTile / 8) {
#pragma unroll
                            for (int u = 4 * g8; u < 4 * g8 + 4; ++u) {
                                float a, b;
                                split_f32(x[u], &a, &b);
                                x[u] = pair_f32(ex2(a), ex2(b));
                            }
                        }
                        if (g8 > 0) {
#pragma unroll
                            for (int u = 4 * g8 - 4; u < 4 * g8; ++u) {
                                float a, b;
                                split_f32(x[u], &a, &b);
                                sum2[u & 1] = add_f32x2(sum2[u & 1], x[u]);
                                w[u] = pack16<BF16>(a, b);
                            }
                            if (g8 % 4 == 0) tmem_st_16(t_s + (g8 / 4 - 1) * 16, w + (g8 / 4 - 1) * 16);
                            if (g8 == kTile / 16 + 2) {  // by now the first half of P has been written: its products may start
                                tmem_wait_st();
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&ctl->p_half[s]);
                            }
                        }
                    }
                    float sum[4];
                    split_f32(sum2[0], &sum[0], &sum[1]);
                    split_f32(sum2[1], &sum[2], &sum[3]);
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (!warp_real) mbar_arrive(&ctl->p_half[s]);
                    mbar_arrive(&ctl->p_ready[s]);
                }
            }
            base += nt;
            if (!ok) break;
            // the O that this thread reads: its stream's, or (a query tile over two streams) both
            if (PAIR) {
                if (nt > 0) ok = warp_wait(ctl, &ctl->o_full[s], n_o0++ & 1, c, g.tries);
            } else {
                if (nt > 0) ok = warp_wait(ctl, &ctl->o_full[0], n_o0++ & 1, c, g.tries);
                if (ok && nt > 1) ok = warp_wait(ctl, &ctl->o_full[1], n_o1++ & 1, c, g.tries);
            }
            if (!ok) break;
            tc_fence_after();
            // ---- the segment's result: this thread's columns [c0, c1) of row r ----
            constexpr int kCols = PAIR ? D : D / 2;
            const int c0 = PAIR ? 0 : s * kCols;
            float keep0 = 1.f, keep1 = 0.f;  // factors of the two streams' O
            bool use0 = steps > 0, use1 = false;
            if (!PAIR) {
                ctl->max_sum[s][0][r] = m;
                ctl->max_sum[s][1][r] = l;
                mbar_arrive(&ctl->sync[0]);
                if (!(ok = warp_wait(ctl, &ctl->sync[0], n_sync & 1, c, g.tries))) break;
                ++n_sync;
                const float m0 = ctl->max_sum[0][0][r], m1 = ctl->max_sum[1][0][r];
                m = fmaxf(m0, m1);
                keep0 = m0 == -INFINITY ? 0.f : ex2((m0 - m) * sc);
                keep1 = m1 == -INFINITY ? 0.f : ex2((m1 - m) * sc);
                l = ctl->max_sum[0][1][r] * keep0 + ctl->max_sum[1][1][r] * keep1;
                use0 = nt > 0;
                use1 = nt > 1;
            }
            const bool whole = seg.first == 0 && seg.last == seg.tiles;
            int cf = 0, cl = 0;
            float *slot = nullptr;
            if (!whole) {
                cf = seg.cf;
                cl = seg.cl;
                const size_t index = (size_t(blockIdx.x) * 2 + (static_cast<int>(blockIdx.x) == cf ? 1 : 0)) * S::QT + (PAIR ? s : 0);
                slot = g.partials + index * S::kSlotFloats;
            }
            uint32_t out_head = 0;
            unsigned short *out = nullptr;
            if (real) {
                out_head = seg.kv_head * g.group + row_head;
                out = static_cast<unsigned short *>(g.out) + static_cast<long long>(seg.q0 + token) * g.out_token +
                      static_cast<long long>(out_head) * g.out_head;
            }
            const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // NaN stays
            // Four lanes exchange their rows' quarters of 32 columns, so that a store instruction writes 64 bytes of each of eight rows
            // instead of 16 of each of 32.
            unsigned long long row_to[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) row_to[k] = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), (lane & ~3) + k);
            if (warp_real) {
#pragma unroll 1
                for (int q = 0; q < kCols / 32; ++q) {
                    float o[32];
                    if (PAIR) {
                        uint32_t a[32];
                        tmem_ld_32(t_o + q * 32, a);
                        tmem_wait_ld();
#pragma unroll
                        for (int u = 0; u < 32; ++u) o[u] = use0 ? __uint_as_float(a[u]) : 0.f;
                    } else {
                        uint32_t a[32], b[32];
                        const uint32_t col = tmem + 2 * kTile + lanes + c0 + q * 32;
                        tmem_ld_32(col, a);
                        tmem_ld_32(col + kTile, b);
                        tmem_wait_ld();
#pragma unroll
                        for (int u = 0; u < 32; ++u)
                            o[u] = (use0 ? __uint_as_float(a[u]) * keep0 : 0.f) + (use1 ? __uint_as_float(b[u]) * keep1 : 0.f);
                    }
                    if (whole) {
                        uint32_t w[4][4];
#pragma unroll
                        for (int u = 0; u < 16; ++u) w[u / 4][u % 4] = pack16<BF16>(o[2 * u] * inv, o[2 * u + 1] * inv);
                        transpose_4(w, lane);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (row_to[k] != 0)
                                *reinterpret_cast<uint4 *>(reinterpret_cast<unsigned short *>(row_to[k]) + c0 + q * 32 + (lane & 3) * 8) =
                                    make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
                    } else if (real) {
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            __stcg(reinterpret_cast<float4 *>(slot) + ((c0 + q * 32) / 4 + u) * kTile + r,
                                   make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]));
                    }
                }
            }
            if (whole) {
                if (real && g.lse && (PAIR || s == 0))
                    g.lse[static_cast<size_t>(seg.q0 + token) * (c.kv_heads * g.group) + out_head] =
                        log_sum<BF16>(m * sc, l);
                if (!PAIR) {  // the other stream's O has been read before it is written again
                    mbar_arrive(&ctl->sync[0]);
                    if (!(ok = warp_wait(ctl, &ctl->sync[0], n_sync & 1, c, g.tries))) break;
                    ++n_sync;
                }
                continue;
            }
            // ---- an item cut by ranges' ends: the last of its blocks joins the partial results ----
            // Where that is more data than one SM should read, in two steps: groups of neighbouring blocks' parts first.
            if (real && (PAIR || s == 0)) {
                __stcg(slot + size_t(kTile) * D + r, m);
                __stcg(slot + size_t(kTile) * (D + 1) + r, l);
            }
            const int first_token = seg.tile * step + (PAIR ? s * g.tile_tokens : 0);
            const int rows = min(g.tile_tokens, seg.n - first_token) * g.group;  // may be <= 0: the second tile of a pair
            const int shift = rows > 1 ? 32 - __clz(rows - 1) : 0;
            auto join = [&](auto steps) {  // whether its waits ended well
                constexpr bool TWO = decltype(steps)::value == 2;
                constexpr unsigned kSlot = static_cast<unsigned>(S::QT * S::kSlotFloats), kBlock = 2 * kSlot;
                int first = cf, span = 2;  // first block of the parts
                Join j;
                j.stride = kBlock;
                j.count = cl - cf + 1;
                j.max_col = D;
                bool final = !TWO;
                if (TWO) {
                    while (span * span < j.count) ++span;
                    first += (static_cast<int>(blockIdx.x) - cf) / span * span;
                    j.count = min(span, cl + 1 - first);
                }
                for (;; final = true) {
                    __threadfence();
                    uint64_t *sync = &ctl->sync[PAIR ? s : 0];
                    mbar_arrive(sync);
                    if (!warp_wait(ctl, sync, n_sync & 1, c, g.tries)) return false;
                    ++n_sync;
                    if (r == 0 && (PAIR || s == 0)) {
                        // a byte for each stream's arrivals at a first and at the last join
                        unsigned *count = g.arrivals + first * 2 + (first == cf ? 1 : 0);
                        const unsigned at = (PAIR ? s * 16 : 0) + (j.stride != kBlock ? 8 : 0);
                        const bool is_last = ((atomicAdd(count, 1u << at) >> at) & 255u) + 1u == static_cast<unsigned>(j.count);
                        ctl->last[PAIR ? s : 0] = is_last;
                        __threadfence();
                        if (is_last) atomicSub(count, static_cast<unsigned>(j.count) << at);
                    }
                    mbar_arrive(sync);
                    if (!warp_wait(ctl, sync, n_sync & 1, c, g.tries)) return false;
                    ++n_sync;
                    if (!ctl->last[PAIR ? s : 0] || rows <= 0) return true;
                    j.base = g.partials + (PAIR ? s : 0) * S::kSlotFloats + static_cast<unsigned>(first) * kBlock;
                    j.lead = first == cf ? kSlot : 0;
                    // A thread keeps to one row and takes its columns, four at a time, in strides.
                    constexpr int kJoiners = PAIR ? 128 : 256;
                    const int joiner = PAIR ? r : s * kTile + r;
                    const int my_row = joiner & ((1 << shift) - 1), c4_step = kJoiners >> shift;
                    const int row = min(my_row, rows - 1);  // the threads beyond the rows only load
                    float top = -INFINITY, z = 0.f;
                    for (int k0 = 0; k0 < j.count; k0 += 8) {
                        float pm[8], pl[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            pm[u] = -INFINITY, pl[u] = 0.f;
                            if (k0 + u < j.count) {
                                const float *p = j.part(k0 + u) + size_t(kTile) * j.max_col + row;
                                pm[u] = __ldcg(p);
                                pl[u] = __ldcg(p + kTile);
                            }
                        }
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const float up = fmaxf(top, pm[u]);
                            const float k = pm[u] == -INFINITY ? 0.f : ex2((pm[u] - up) * sc);
                            z = z * (top == -INFINITY ? 0.f : ex2((top - up) * sc)) + pl[u] * k;
                            top = up;
                        }
                    }
                    const int tk = row / g.group, hd = seg.kv_head * g.group + row - tk * g.group;
                    const long long qt = seg.q0 + first_token + tk;
                    const float f = z > 0.f ? 1.f / z : z == 0.f ? 0.f : z;
                    unsigned short *to = static_cast<unsigned short *>(g.out) + qt * g.out_token + hd * g.out_head;
                    if ((joiner >> shift) == 0 && my_row == row) {
                        if (!final) {
                            float *p = j.part(0) + size_t(kTile) * (D + 2) + row;
                            __stcg(p, top);
                            __stcg(p + kTile, z);
                        } else if (g.lse) {
                            g.lse[qt * (c.kv_heads * g.group) + hd] = log_sum<BF16>(top * sc, z);
                        }
                    }
                    const int c4 = my_row == row ? joiner >> shift : D / 4;
                    // Eight to sixteen vectors in flight a thread: two parts are the rule where query tiles fill their rows; with few rows
                    // there may be many parts.
                    if (PAIR)
                        join_columns<BF16, D, 8, 2>(j, row, c4, c4_step, top, f, sc, final, to);
                    else if (c4_step * 2 <= D / 4)
                        join_columns<BF16, D, 4, 2>(j, row, c4, c4_step, top, f, sc, final, to);
                    else
                        join_columns<BF16, D, 1, 16>(j, row, c4, c4_step, top, f, sc, final, to);
                    if (!TWO || final) return true;
                    first = cf;
                    j.stride = span * kBlock;
                    j.count = (cl - cf) / span + 1;
                    j.max_col = D + 2;
                }
            };
            ok = ((cl - cf + 1) << shift) < kTwoSteps ? join(std::integral_constant<int, 1>()) : join(std::integral_constant<int, 2>());
            if (!ok) break;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, kTmemCols);
}

template <bool BF16, int D, bool PAIR>
dspark_status launch(const CUtensorMap &tm_q, const CUtensorMap &tm_kv, const CacheView &c, const Attention &g, int blocks,
                     cudaStream_t stream) {
    auto *kernel = attention_kernel<BF16, D, PAIR>;
    static int configured = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (configured != dev) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(paged_attention)");
        // the register shares are taken from what the block is launched with: never ask for more
        cudaFuncAttributes attr;
        e = cudaFuncGetAttributes(&attr, kernel);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes(paged_attention)");
        if (attr.numRegs < kLaunchRegs) return fail(DSPARK_ERR_CUDA, "paged_attention: built with %d registers a thread", attr.numRegs);
        configured = dev;
    }
    e = launch_pdl(kernel, dim3(blocks), dim3(kThreads), kSmemBytes, stream, tm_q, tm_kv, c, g);
    return e == cudaSuccess ? DSPARK_OK : cuda_fail(e, "paged_attention");
}

dspark_status attend(const dspark_cache *cache, const dspark_attention_args *args, unsigned stall_us, cudaStream_t stream) {
    const char *who = "paged_attention";
    CacheView c;
    dspark_status st = cache_view(cache, who, &c);
    if (st != DSPARK_OK) return st;
    if (!args) return fail(DSPARK_ERR_INVALID, "%s: null arguments", who);
    auto [q, out, lse, rows, cu_new, q_token_stride, q_head_stride, out_token_stride, out_head_stride, layer, tokens, q_heads, n_seqs,
          max_new, causal, window, scale] = *args;
    if (layer < 0 || layer >= c.layers) return fail(DSPARK_ERR_INVALID, "%s: layer %d of %d", who, layer, c.layers);
    if (tokens < 0 || q_heads < 1 || n_seqs < 0 || max_new < 0 || window < 0)
        return fail(DSPARK_ERR_INVALID, "%s: bad sizes tokens=%d q_heads=%d n_seqs=%d max_new=%d window=%d", who, tokens,
                    q_heads, n_seqs, max_new, window);
    if (q_heads % c.kv_heads) return fail(DSPARK_ERR_INVALID, "%s: %d query heads over %d kv heads", who, q_heads, c.kv_heads);
    if (!(scale > 0.f) || scale > 3.0e38f) return fail(DSPARK_ERR_INVALID, "%s: scale %g is not positive and finite", who, scale);
    const int group = q_heads / c.kv_heads;
    if (group > kTile) return fail(DSPARK_ERR_UNSUPPORTED, "%s: %d query heads to a kv head, at most %d", who, group, kTile);
    if (n_seqs > kMaxSeqs) return fail(DSPARK_ERR_UNSUPPORTED, "%s: n_seqs %d > %d", who, n_seqs, kMaxSeqs);
    if (tokens == 0 || n_seqs == 0) return DSPARK_OK;
    if (!q || !out || !cu_new) return fail(DSPARK_ERR_INVALID, "%s: null pointer argument", who);
    // strides of axes of one entry are never used: any value will do
    if (tokens == 1) q_token_stride = out_token_stride = static_cast<long long>(q_heads) * c.head_dim;
    if (q_heads == 1) q_head_stride = out_head_stride = c.head_dim;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cu_new, 4) || !aligned(lse, 4) || q_token_stride % 8 ||
        q_head_stride % 8 || out_token_stride % 8 || out_head_stride % 8 || q_token_stride <= 0 || q_head_stride <= 0 ||
        out_token_stride < 0 || out_head_stride < 0)
        return fail(DSPARK_ERR_INVALID, "%s: q and out must be 16-byte aligned, with positive strides of whole 16 bytes", who);
    int sms = 0;
    if ((st = static_cast<dspark_status>(current_sm_count(&sms))) != DSPARK_OK) return st;
    // The kernel counts key tiles in 32 bits: at most one item for each token and sequence of a kv head, of all the tiles of a row.
    const double items = (static_cast<double>(tokens) / (kTile / group) + n_seqs) * c.kv_heads;
    if (items * (static_cast<double>(c.max_pages) * c.page_size / kTile + 1 + kItemCost) > 4.0e9)
        return fail(DSPARK_ERR_UNSUPPORTED, "%s: %d tokens of %d sequences over rows of %d pages pass 2^32 key tiles", who, tokens, n_seqs,
                    c.max_pages);

    const cuuint64_t page_groups = 2ull * c.layers * c.kv_heads * (c.page_size / 8), groups = page_groups * c.num_pages;
    if (groups + page_groups > 0x7fffffffull)
        return fail(DSPARK_ERR_UNSUPPORTED, "%s: a pool of more than 2^31 groups of 8 slots of a head", who);

    Attention g{};
    g.out = out;
    g.lse = lse;
    g.out_token = out_token_stride;
    g.out_head = out_head_stride;
    g.rows = rows;
    g.cu_new = cu_new;
    g.tokens = tokens;
    g.group = group;
    g.n_seqs = n_seqs;
    g.layer = layer;
    g.causal = causal != 0;
    g.window = window < 1 << 30 ? window : 0;  // no row is longer: hides nothing, and differences of positions stay within 32 bits
    g.scale = scale;
    g.tile_tokens = kTile / group;
    // Two query tiles share each key tile where chunks have two; a chunk of one tile splits its keys over the streams. Query tiles
    // in pairs against one at a time: 16 chunks of 33 tokens (a tile holds 32) over 3000 keys 52 against 77 us, of 96
    // tokens 92 against 110, 8192 tokens after 8192 1019 against 1147; of chunks that one tile holds, 1-8 tokens over 16,000-66,000
    // keys 200 against 182. Four chunks of 64 tokens are the exception (35 against 29): few items, so more blocks join each.
    const bool pair = max_new > g.tile_tokens;
    const int step = g.tile_tokens * (pair ? 2 : 1);
    g.chunk_tiles = (max_new + step - 1) / step;
    // Partial sums, their join and the walk between items take as long as some key tiles, the more rows the more. Every item whole |
    // all cut into equal ranges: 32 tokens over 1000 keys 13.7 | 17.3 us, 400 tokens of 2 sequences 12.9 | 35.1, 1024 after 4000
    // 62.9 | 67.9; 9 key tiles of one token 12.0 | 10.8, 17 of 7 tokens 17.8 | 12.1, 4 chunks of 64 tokens over 3000 keys 39.2 | 34.8.
    g.cut = pair || max_new * group >= kTile ? 16 : 6 + 6 * max_new * group / kTile;
    g.partials = reinterpret_cast<float *>(c.scratch);
    g.arrivals = c.counters;
    g.timeout_ns = kDefaultTimeoutNs;
    g.tries = static_cast<uint32_t>(kDefaultTimeoutNs / 1000);
    g.stall_ns = static_cast<unsigned long long>(stall_us) * 1000ull;

    const bool bf16 = cache->dtype == DSPARK_BF16;
    CUtensorMap tm_q, tm_kv;
    {
        const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(q_heads), static_cast<cuuint64_t>(tokens)};
        const cuuint64_t strides[2] = {static_cast<cuuint64_t>(q_head_stride) * 2, static_cast<cuuint64_t>(q_token_stride) * 2};
        const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(g.tile_tokens)};
        if ((st = make_tmap_nd(&tm_q, bf16, q, 3, dims, strides, box)) != DSPARK_OK) return st;
    }
    {
        // all of the pool as groups of 8 slots of one page, layer, half and head
        const cuuint64_t dims[4] = {64, 8, static_cast<cuuint64_t>(c.head_dim / 64), groups};
        const cuuint64_t strides[3] = {2ull * c.head_dim, 128, 16ull * c.head_dim};
        const cuuint32_t box[4] = {64, 8, static_cast<cuuint32_t>(c.head_dim / 64),
                                   static_cast<cuuint32_t>((c.page_size < kTile ? c.page_size : kTile) / 8)};
        if ((st = make_tmap_nd(&tm_kv, bf16, c.pool, 4, dims, strides, box)) != DSPARK_OK) return st;
    }
    const int blocks = sms < kMaxCtas ? sms : kMaxCtas;
    auto *run = c.head_dim == 128 ? (bf16 ? (pair ? launch<true, 128, true> : launch<true, 128, false>)
                                          : (pair ? launch<false, 128, true> : launch<false, 128, false>))
                                  : (bf16 ? (pair ? launch<true, 64, true> : launch<true, 64, false>)
                                          : (pair ? launch<false, 64, true> : launch<false, 64, false>));
    return run(tm_q, tm_kv, c, g, blocks, stream);
}

}  // namespace

// Two slots a block, of two query tiles each.
size_t attention_scratch_bytes(int head_dim) { return size_t(kMaxCtas) * 2 * 2 * slot_bytes(head_dim); }

}  // namespace dspark

extern "C" dspark_status dspark_paged_attention(const dspark_cache *cache, const dspark_attention_args *args, dspark_stream_t stream) {
    return dspark::attend(cache, args, 0, stream);
}

extern "C" dspark_status dspark_paged_attention_debug(const dspark_cache *cache, const dspark_attention_args *args, unsigned stall_us,
                                                      dspark_stream_t stream) {
    return dspark::attend(cache, args, stall_us, stream);
}
