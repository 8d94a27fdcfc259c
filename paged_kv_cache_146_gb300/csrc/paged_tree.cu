// Attention of trees of drafted tokens over the paged cache (sm_103a).
//
// Row r, drafted token i of its sequence (context L, n drafted tokens, base = L - n):
//   x_j = scale <q, K_j>,  out = sum_j softmax(x)_j V_j   over the j that it sees:
//   j < base,  or  base <= j < L and bit j - base of its mask is set.
//
// All n G rows of a (sequence, kv head) share its keys: K and V are read once for each query
// tile of up to 128 rows, one row to a lane of tensor memory, and both products run on
// tcgen05.  An item is a query tile of a (sequence, kv head); the key tiles (64 keys) of all items,
// written one after the other with kItemCost tiles' worth of overhead before each, are cut into
// equal ranges, one to a CTA: every CTA has the same work, whatever the lengths, and an item is
// cut where a range ends.  A cut item's pieces (unnormalised output, reference, sum; fp32) meet
// in the workspace and a second kernel joins them, always in the same order.
//
// Items go first query tiles first, by sequence and kv head, then the second ones, and so on:
// where trees need two tiles, two CTAs read the same keys at about the same time, one of
// them from L2.  Two CTAs fit an SM, with 256 columns of tensor memory each; while one waits for
// its softmax or begins an item, the other keeps copies and products going (96 long sequences
// 795 us with one CTA, 554 with two, then).
//
// What bounds it, 32 query heads over 8 of 128: at 96 sequences of up to 16,384 tokens with 16
// drafted ones the copies of K and V (3.43 GB in 511-556 us, 6.2-6.7 TB/s; a plain copy's
// rate is 6.8).  At 24 sequences with 64 drafted, two full query tiles each, nothing alone (140-156 us
// by machine; the bytes 70, the products 59): the main kernel's 128 us bring every key tile twice
// (7.4 TB/s from L2), keep the tensor pipe busy for 58 % (P V once for each part of the weights), and
// the softmax warps wait for fixed latencies; 15 us go to joining 39 MB of pieces.  A second tile
// that is partly full costs as much as a full one: 64 sequences of 33 drafted tokens behind 500
// 62 us, three times their bytes.  At 4 sequences, 22 us, the chain of lengths -> plan -> block ids ->
// tiles -> pieces -> joining kernel (the bytes 6).  Heads of 64: a key tile is half the bytes, the chain
// as long (29 sequences of 40 heads 90 us, the bytes 63).
//
// Roles of a CTA's warps:
//   0-3, softmax: thread r owns row r.  Weights are taken against a lazy reference (it moves
//     when a score exceeds it by more than kLazy, in log2 units), as two 16-bit parts each,
//     into tensor memory.  Every kFlush tiles O goes to a sum in the workspace.
//   4, producer: makes the plan and hands out the items; a ring of K tiles and one of V tiles,
//     one TMA box to each block and 64 columns; the items' query rows.
//   5, issuer: S = Q K^T into one of two buffers, then O += P V of the tile before.
//   6, cleaner: V of keys that no row may be reached by.  A weight of zero does not stop a NaN
//     or an infinity in V, so in tiles that hold drafted tokens or the end of the sequence V
//     behind the end becomes zero, and so do V's odd values; rows that see such a key get
//     them added by hand (rare).
// Every wait is bounded; on expiry the kernel flags PKV_DEV_TIMEOUT and stops.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <mutex>

#include "pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tc_device.cuh"

namespace pkv {
namespace tree {

constexpr int kRows = 128;             // M: rows of a query tile
constexpr int kKeys = 64;              // keys of a tile
constexpr int kMaxWords = 32;
constexpr int kTilesKnown = 16;        // tiles whose bad blocks are remembered
constexpr int kTasks = 8;              // items under way, at most
constexpr int kAhead = 2;              // lengths of so many 32 sequences are read at once
constexpr float kLazy = 8.f;
// An item's beginning and end, in tiles (20 ragged sequences of 40 kv heads: 94 us, 125 when items
// cost nothing, 95 when 4), and the shortest piece that is cut off an item (24 sequences of 64
// drafted tokens: 143 us, 147 with 1; the 40 heads 97 with 4).
constexpr int kItemCost = 2, kSnap = 2;
constexpr int kMaxRanges = 304;        // CTAs of a call, at most
// Tiles after which O is moved to a sum in the workspace.  The tensor cores' additions into O
// truncate, so O falls behind by some 2^-23 of itself with every matrix instruction: 131,072 tokens of
// positive values came out 1.1e-3 low, twice the half step of fp16, 16,384 2e-4.  Moved every 128
// tiles it is 1e-4 whatever the length, and the sums of the moved ones round.  (96 sequences of up
// to 16,384 tokens 528 -> 534 us; every 64 tiles 5e-5 and 539.  Without the hint that keeps the
// sums in L2 545 and 557.)
constexpr int kFlush = 128;

struct Params {
    void *out;
    const void *v_pool;
    const int32_t *block_tables, *query_start, *context_lens;
    const uint32_t *mask;
    int32_t words, num_seqs, num_tokens, num_q_heads, num_kv_heads, group;
    int32_t max_blocks_per_seq, num_blocks;
    int32_t max_tokens;                // that a table row holds
    int32_t tile_tokens;               // tokens of a query tile
    int32_t box_tokens;                // and of one box of query rows
    int32_t tile_inverse;              // ceil(2^20 / tile_tokens)
    int32_t piece_rows;                // rows of a piece's place in the workspace
    float scale_log2;                  // > 0
    int32_t negate;                    // the scale is negative
    int32_t grid;                      // CTAs of the call
    int4 *ranges;                      // [grid], see kContinues
    float2 *part_ml;                   // [2 ranges][piece_rows]: (reference, sum); sum < 0: bad block
    float4 *part_o;                    // [2 ranges][D / 4][piece_rows]
    int32_t *status;
};

// What CTA b leaves for the joining kernel: x = 1 it holds the continuation of an item that began
// in an earlier range (piece 2 b), + 2 up to the item's end, + 4 it begins an item that ends in a
// later range (piece 2 b + 1), of y tokens from row z on, kv head w; + 8 in every range where some
// sequence's lengths do not fit: the joining kernel makes its rows zero.
constexpr int kContinues = 1, kEnds = 2, kBegins = 4, kRefused = 8;

// One sequence of a call.
struct Seq {
    int r0, n, base, L, tiles, parts;  // rows; key tiles; query tiles
    bool rows_ok, bad;
};

__device__ __forceinline__ Seq seq_of(const Params &p, int r0, int r1, int L)
{
    Seq q;
    q.r0 = r0;
    q.L = L;
    q.rows_ok = 0 <= q.r0 && q.r0 <= r1 && r1 <= p.num_tokens;
    q.n = q.rows_ok ? r1 - q.r0 : 0;
    q.bad = !q.rows_ok || q.L < q.n || q.L > p.max_tokens || q.n > 32 * p.words;
    q.base = q.L - q.n;
    q.tiles = (q.L + kKeys - 1) / kKeys;
    // ceil(n / tile_tokens): n + tile_tokens < 1280 here, so 2^20 is enough for the inverse
    q.parts = q.bad ? 0 : (q.n + p.tile_tokens - 1) * p.tile_inverse >> 20;
    return q;
}

// A place in the order of all tiles: key tile t of query tile k of sequence s and kv head g.
struct Place {
    int k, s, g, t;
    // the items that the places are in
    __device__ __forceinline__ bool operator==(const Place &o) const { return k == o.k && s == o.s && g == o.g; }
    __device__ __forceinline__ bool operator<(const Place &o) const
    {
        return k != o.k ? k < o.k : s != o.s ? s < o.s : g < o.g;
    }
};

// An item's part in a range: tiles [t0, t1) of kv head g and the query tiles from token `first`
// on, of sequence s.  t0 == t1: there are no more.
struct alignas(16) Task {
    int s, g, first, t0, t1;
    int r0, n, base;                   // the sequence's rows, drafted tokens and tokens before them
    __device__ __forceinline__ int L() const { return base + n; }
};

// The place where a range ends that would end `off` units into sequence s's: not inside an
// item's overhead, and not so near an end of the item that a short piece would be left.
// (Leaving short items whole where a cut's pieces cost more bytes than it saves made no case
// faster: 24 trees of 64 157 -> 176 us, 12 sequences of 16 heads 17 -> 27.)
__device__ __forceinline__ Place cut(const Params &p, int k, int s, const Seq &q, uint32_t off, int snap)
{
    const uint32_t per = q.tiles + kItemCost;
    Place c = {k, s, (int)(off / per), 0};
    const int t = (int)(off - c.g * per) - kItemCost;
    c.t = t < snap ? 0 : t;
    if (t > q.tiles - snap) {
        c.t = 0;
        if (++c.g == p.num_kv_heads) {
            c.g = 0;
            ++c.s;
        }
    }
    return c;
}

// A CTA's range and the way through its items; the producer's warp makes it and goes it for the
// CTA.  Lane i holds the lengths of sequence `held` + i.  (The host sees to it that all units of a
// call fit 32 bits.)
struct Walk {
    Place at, to;
    Seq q;                             // sequence at.s
    int most;                          // query tiles of a sequence, at most
    int held, r0, r1, L;

    __device__ __forceinline__ void hold(const Params &p, int s)
    {
        held = s;
        const int i = s + (int)(threadIdx.x & 31);
        r0 = i < p.num_seqs ? p.query_start[i] : 0;
        r1 = i < p.num_seqs ? p.query_start[i + 1] : 0;
        L = i < p.num_seqs ? p.context_lens[i] : 0;
    }
    __device__ __forceinline__ Seq sequence(const Params &p, int i) const
    {
        return seq_of(p, __shfl_sync(kFull, r0, i), __shfl_sync(kFull, r1, i), __shfl_sync(kFull, L, i));
    }

    // The ranges: the units of all sequences are counted, and the two ends of this CTA's range
    // looked up.  CTA s % gridDim also reports sequences whose lengths do not fit.
    __device__ __forceinline__ void plan(const Params &p)
    {
        const int lane = threadIdx.x & 31;
        // of one query tile
        auto units_of = [&](const Seq &x) { return (uint32_t)p.num_kv_heads * (uint32_t)(x.tiles + kItemCost); };
        uint32_t all = 0;
        most = 0;
        bool refused = false;
#pragma unroll 1
        for (int s0 = 0; s0 < p.num_seqs; s0 += 32 * kAhead) {
            int a[kAhead], b[kAhead], len[kAhead];       // the loads of several steps at once
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = s0 + 32 * k + lane;
                a[k] = i < p.num_seqs ? p.query_start[i] : 0;
                b[k] = i < p.num_seqs ? p.query_start[i + 1] : 0;
                len[k] = i < p.num_seqs ? p.context_lens[i] : 0;
            }
            held = s0;
            r0 = a[0];
            r1 = b[0];
            L = len[0];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const Seq x = seq_of(p, a[k], b[k], len[k]);
                all += x.parts * units_of(x);
                most = max(most, x.parts);
                refused |= x.bad;
                if (x.bad && (s0 + 32 * k + lane) % gridDim.x == blockIdx.x) atomicOr(p.status, PKV_DEV_BAD_LEN);
            }
        }
        refused = __any_sync(kFull, refused);
        all = __reduce_add_sync(kFull, all);
        most = __reduce_max_sync(kFull, most);
        const uint32_t ranges = max(1u, min(gridDim.x, all));
        // range b begins at all b / ranges: the rest is spread evenly, so that CTAs at the same
        // place among first and among second query tiles keep in step
        const uint32_t size = all / ranges, more = all - size * ranges;
        const int snap = min(kSnap, (int)(size / 4));
        const uint32_t begin = size * blockIdx.x + more * blockIdx.x / ranges;
        const uint32_t end = size * (blockIdx.x + 1) + more * (blockIdx.x + 1) / ranges;
        at = to = Place{most, 0, 0, 0};
        int4 left = make_int4(refused ? kRefused : 0, 0, 0, 0);          // for the joining kernel
        uint32_t before = 0;
#pragma unroll 1
        for (int k = 0; k < most && blockIdx.x < ranges && before <= end; ++k) {
#pragma unroll 1
            for (int s0 = 0; s0 < p.num_seqs && before <= end; s0 += 32) {
                if (s0 != held) hold(p, s0);
                const Seq mine = seq_of(p, r0, r1, L);
                const uint32_t units = mine.parts > k ? units_of(mine) : 0u;
                uint32_t upto = units;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(kFull, upto, o);
                    if (lane >= o) upto += y;
                }
#pragma unroll 1
                for (int e = 0; e < 2; ++e) {
                    const uint32_t off = (e ? end : begin) - before;         // (wraps below `before`)
                    const unsigned who = __ballot_sync(kFull, off >= upto - units && off < upto);
                    if (!who) continue;
                    const int src = __ffs(who) - 1;
                    const Seq x = sequence(p, src);
                    const Place c = cut(p, k, s0 + src, x, off - __shfl_sync(kFull, upto - units, src), snap);
                    if (!e) {
                        at = c;
                        continue;
                    }
                    to = c;
                    const int first = k * p.tile_tokens;
                    left = make_int4(left.x, min(p.tile_tokens, x.n - first), x.r0 + first, c.g);
                }
                before += __shfl_sync(kFull, upto, 31);
            }
        }
        const bool same = at == to;
        if (at.t > 0) left.x |= kContinues | (same ? 0 : kEnds);
        if (to.t > 0 && !(same && at.t > 0)) left.x |= kBegins;
        if (lane == 0) p.ranges[blockIdx.x] = left;
        if (at.s < held || at.s >= held + 32) hold(p, at.s);
        q = sequence(p, at.s - held);
    }
    __device__ __forceinline__ Task next(const Params &p)
    {
        Task task = {};
        while (at < to || (at == to && at.t < to.t)) {
            if (at.s >= p.num_seqs) {                    // the next query tiles
                ++at.k;
                at.s = at.g = 0;
                hold(p, 0);
                q = sequence(p, 0);
                continue;
            }
            if (q.parts > at.k) {
                task.s = at.s;
                task.g = at.g;
                task.first = at.k * p.tile_tokens;
                task.t0 = at.t;
                task.t1 = at == to ? to.t : q.tiles;
                task.r0 = q.r0;
                task.n = q.n;
                task.base = q.base;
                at.t = 0;
                if (++at.g < p.num_kv_heads) return task;
            }
            at.g = 0;
            if (++at.s < p.num_seqs) {
                if (at.s >= held + 32) hold(p, at.s);
                q = sequence(p, at.s - held);
            }
            if (task.t0 < task.t1) return task;
        }
        return task;
    }
};

__device__ __forceinline__ float max3f(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Product of a hidden key: the scale carries it to -inf (it is never zero, see the host).
constexpr float kHide = -INFINITY;

// One tensor-memory column of this thread's lane.
__device__ __forceinline__ uint32_t column(uint32_t taddr)
{
    uint32_t v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr));
    tc::tmem_wait_ld();
    return v;
}
__device__ __forceinline__ void set_column(uint32_t taddr, uint32_t v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
    tc::tmem_wait_st();
}

// One lane of the warp, always the same.  Code that only it runs, in a branch of the whole warp,
// keeps the operands of matrix instructions and copies in uniform registers; in a branch by
// lane number each operand goes through a move of its own, and the issue of a tile's products
// took as long as its softmax.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// The n lowest of 64 bits (all for n >= 64, none for n <= 0).
__device__ __forceinline__ uint64_t low_bits(int n)
{
    return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull;
}

// Keys k0 .. k0 + 63 that a drafted token sees; `words` its mask, w0 and w1 its first two words.
__device__ __forceinline__ uint64_t seen_keys(const Params &p, const uint32_t *words, uint32_t w0,
                                              uint32_t w1, int k0, int base, int L)
{
    const int d = k0 - base;                     // drafted token of key k0
    const uint64_t two = w0 | (uint64_t)w1 << 32;
    uint64_t bits;
    if (d <= 0) {
        bits = two << -d | low_bits(-d);         // (base - k0 < 64: the tile holds drafted tokens)
    } else if (p.words <= 2) {
        bits = two >> (d & 63);                  // (d < 64: the tile holds a drafted token)
    } else {
        const int w = d >> 5, sh = d & 31;
        const uint64_t a = w < p.words ? words[w] : 0u, b = w + 1 < p.words ? words[w + 1] : 0u;
        const uint64_t c = w + 2 < p.words ? words[w + 2] : 0u;
        bits = (a | b << 32) >> sh;
        if (sh) bits |= c << (64 - sh);
    }
    return bits & low_bits(L - k0);
}

// Weights (p0, p1), pp = the same pair packed, as two 16-bit parts, the even key in the low
// half of each word.  The first part is truncated, the rest rounded: bf16 2^-16, fp16 2^-22 (of
// the weight).  The rest is taken 2^-24 of the first part too large, well within that, so that no
// part is negative, or zero beside another one, as long as 16 bits can hold it: an infinity in V
// times the parts is that infinity, where inf - inf or 0 inf would be NaN.
//
// bf16 stays at two parts: 2^-16 is 2^-8 of what the output's own rounding takes off, and moves one
// value in some hundred by that rounding's step (1.4e-4 of a result's norm; its error against 64
// bits is the same, 1.66e-3).  A third part (2^-24; 0.9e-4 on 4 sequences, no gain on long contexts,
// where it is the sums' rounding) is half as many products again and has no place in tensor memory;
// with it in shared memory 96 long sequences took 604-630 us in place of 512-528, 24 x 64 168-176 in
// place of 140-143, and as much where it borrowed the next tile's columns.
constexpr float kRest = -(1.f - 0x1p-24f);
template <bool BF16>
__device__ __forceinline__ void two_parts(float p0, float p1, uint64_t pp, uint32_t &hi, uint32_t &lo)
{
    float2 h;
    if constexpr (BF16) {
        const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
        hi = __byte_perm(b0, b1, 0x7632);
        h = make_float2(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u));
    } else {
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(p1), "f"(p0));
        h = Elem<false>::unpack(hi);
    }
    const float2 d = unpack2f(fma2f(pack2f(h.x, h.y), pack2f(kRest, kRest), pp));
    lo = Elem<BF16>::pack(d.x, d.y);
}

// One of a word's two values is an infinity or a NaN: their halves as a mask.
template <bool BF16>
__device__ __forceinline__ uint32_t odd_halves(uint32_t w)
{
    constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
    return ((w & kExp) == kExp ? 0xffffu : 0u) | ((w >> 16 & kExp) == kExp ? 0xffff0000u : 0u);
}

// The sum with 0 w added: NaN from the first infinity or NaN on.
template <bool BF16>
__device__ __forceinline__ void add_odd(uint32_t &sum, uint32_t w)
{
    if constexpr (BF16) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(w), "r"(0u));
    else asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(w), "r"(0u));
}

// The row's sum of the tiles before the last kFlush ones lies in the workspace, in the place of the
// item's piece (an item that is not cut uses the later one: the cut item that fills it comes last).
// O, of reference ref, is added to it and cleared, or (back) it is added to O; `any`: there is
// something in it.  The whole warp calls it; as a function it leaves the loop's code alone (inlined,
// calls that never come here took 8 % longer).
template <int D>
__device__ __noinline__ void move_sum(const Params &p, uint32_t t_o, bool begins, bool valid, bool any,
                                      float sum_ref, float ref, bool back)
{
    const int64_t rows = p.piece_rows;
    float4 *sum = p.part_o + (2 * blockIdx.x + begins) * (D / 4) * rows + threadIdx.x;
    const float g = sum_ref == kHide ? 0.f : fast_exp2((sum_ref - ref) * p.scale_log2);
    // most references do not move any more: then nothing is read
    const bool plain = !back && any && __all_sync(kFull, !valid || g == 1.f);
    const bool read = any && valid && !plain;
    uint64_t hint;                       // stays in L2 while keys pass through it, until it is read back
    if (back) asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(hint));
    else asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(hint));
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32, sum += 8 * rows) {
        float4 w[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            w[c] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (read)
                asm volatile("ld.relaxed.gpu.global.L2::cache_hint.v4.f32 {%0, %1, %2, %3}, [%4], %5;"
                             : "=f"(w[c].x), "=f"(w[c].y), "=f"(w[c].z), "=f"(w[c].w)
                             : "l"(sum + c * rows), "l"(hint)
                             : "memory");
        }
        uint32_t v[32];
        tc::tmem_ld32(t_o + c0, v);
        tc::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t *x = &v[4 * c];
            float4 *at = sum + c * rows;
            const float4 y = make_float4(__uint_as_float(x[0]) + g * w[c].x, __uint_as_float(x[1]) + g * w[c].y,
                                         __uint_as_float(x[2]) + g * w[c].z, __uint_as_float(x[3]) + g * w[c].w);
            if (plain && valid)          // (only this thread touches these words: always in the same order)
                asm volatile("red.relaxed.gpu.global.add.L2::cache_hint.v4.f32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(at),
                             "f"(y.x), "f"(y.y), "f"(y.z), "f"(y.w), "l"(hint)
                             : "memory");
            else if (!back && valid)
                asm volatile("st.relaxed.gpu.global.L2::cache_hint.v4.f32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(at),
                             "f"(y.x), "f"(y.y), "f"(y.z), "f"(y.w), "l"(hint)
                             : "memory");
            x[0] = back ? __float_as_uint(y.x) : 0u;
            x[1] = back ? __float_as_uint(y.y) : 0u;
            x[2] = back ? __float_as_uint(y.z) : 0u;
            x[3] = back ? __float_as_uint(y.w) : 0u;
        }
        tc::tmem_st32(t_o + c0, v);
    }
    tc::tmem_wait_st();
}

template <int D>
struct Layout {
    static constexpr int kRegions = D / 64;
    // K and V tiles in flight, a ring each (V waits for the softmax, K does not: 24 sequences of
    // 64 drafted tokens 143 us with 2 and 3, 147 with 3 and 2)
    static constexpr int kK = D == 128 ? 2 : 6, kV = D == 128 ? 3 : 6;
    static constexpr int kQBytes = kRegions * kRows * 128;     // a query tile: [region][row][128 B]
    static constexpr int kTileBytes = kRegions * kKeys * 128;  // a K or V tile
    static constexpr int kKRing = kQBytes, kVRing = kKRing + kK * kTileBytes;
    static constexpr int kMisc = kVRing + kV * kTileBytes, kMiscBytes = 1024;
    static constexpr int kTotal = kMisc + kMiscBytes;          // two CTAs to an SM: at most 113 KB
};

// Warps: softmax, copies and products, and one without a role (the register split goes by
// warpgroups).
constexpr int kProducer = 4, kIssuer = 5, kCleaner = 6, kThreads = 256;
// Registers of a thread: the launch gives kLaunchRegs, the copy and issue warpgroup keeps
// kRegsIo and hands the rest to the softmax warpgroup.  A launch with fewer would leave
// setmaxnreg.inc waiting for ever, so the host launches only kernels of exactly kLaunchRegs.
constexpr int kLaunchRegs = 128, kRegsIo = 104, kRegsSoftmax = 152;
static_assert(kRegsSoftmax + kRegsIo == 2 * kLaunchRegs, "register split of the launch");
constexpr uint32_t kColumns = 256;     // tensor memory: S, S, O

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 2)
    tree_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ CUtensorMap tmQ, const Params p)
{
    using E = Elem<BF16>;
    using T = typename E::T;
    using LY = Layout<D>;
    constexpr int NK = LY::kK, NV = LY::kV;
    // fp16 pools take their weights times 2^kTop: they stay within 2^15, and those down to 2^-21 of
    // the largest are normal numbers in fp16 (a row far below a few dominant keys would lose
    // its weights' bits).
    constexpr float kTop = BF16 ? 0.f : 7.f;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + LY::kMisc);
    uint64_t *q_full = bars, *q_empty = bars + 1;
    uint64_t *k_full = bars + 2, *k_empty = k_full + NK;
    uint64_t *v_full = k_empty + NK, *v_empty = v_full + NV, *clean = v_empty + NV;
    // S out; P out; P V done, each for even and odd tiles
    uint64_t *s_full = clean + NV, *p_full = s_full + 2, *o_full = p_full + 2, *done = o_full + 2;
    uint64_t *task_full = done + 1, *task_empty = task_full + kTasks;
    uint64_t *odd_keys = task_empty + kTasks;            // [NV]: keys whose V held odd values
    // a tile has a bad block: a K tile's slot is free once S is out, before the softmax reads this,
    // so these have places of their own, more than there are tiles under way
    uint8_t *bad_blocks = reinterpret_cast<uint8_t *>(odd_keys + NV);   // [kTilesKnown]
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bad_blocks + kTilesKnown);
    volatile int *abort_flag = reinterpret_cast<int *>(tslot + 1);
    Task *tasks = reinterpret_cast<Task *>(smem + LY::kTotal) - kTasks;
    static_assert((9 + 2 * NK + 4 * NV + 2 * kTasks) * 8 + kTilesKnown + 8 + kTasks * sizeof(Task) <=
                          LY::kMiscBytes && NK + 3 <= kTilesKnown && NV + 3 <= kTilesKnown,
                  "barriers and flags");

    if (smem_addr(smem) & 1023u) {       // the swizzle's atoms; no launch has been seen to do this
        griddep_wait();
        if (threadIdx.x == 0) {
            atomicOr(p.status, PKV_DEV_TIMEOUT);
            p.ranges[blockIdx.x] = make_int4(0, 0, 0, 0);        // nothing to join
        }
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(smem_addr(q_full), 1);
        mbar_init(smem_addr(q_empty), 1);
        for (int i = 0; i < NK; ++i) {
            mbar_init(smem_addr(&k_full[i]), 1);
            mbar_init(smem_addr(&k_empty[i]), 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(smem_addr(&v_full[i]), 1);
            mbar_init(smem_addr(&v_empty[i]), 1);
            mbar_init(smem_addr(&clean[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&s_full[i]), 1);
            mbar_init(smem_addr(&p_full[i]), 4);
            mbar_init(smem_addr(&o_full[i]), 1);
        }
        mbar_init(smem_addr(done), 1);
        for (int i = 0; i < kTasks; ++i) {
            mbar_init(smem_addr(&task_full[i]), 1);
            mbar_init(smem_addr(&task_empty[i]), 6);        // softmax warps, issuer, cleaner
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tc::tmem_alloc(tslot, kColumns);
    if (warp == 1 && lane < 3) {
        const CUtensorMap *map = lane == 0 ? &tmK : lane == 1 ? &tmV : &tmQ;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tslot;
    // a launch may overlap the end of the kernel before it, and the joining kernel the end
    // of this one
    griddep_launch_dependents();
    griddep_wait();
    const int Hkv = p.num_kv_heads, G = p.group, QT = p.tile_tokens;

    // (the register split is taken inside each role's branch, so that all of a role's code
    // lies under one limit)
    uint32_t nt = 0;                     // items that this role has taken
    // A wait of the whole warp, false for all lanes once it ran out for one: each lane looks at the
    // barrier, the flag and the clock by itself, and lanes that went on without the others would
    // leave these at the warp's next vote.
    auto reach = [&](uint64_t *bar, uint32_t parity) {
        return (bool)__all_sync(kFull, mbar_wait(smem_addr(bar), parity, abort_flag, p.status));
    };
    // the next item's task, false once there is none or a wait ran out
    Task it;
    auto next_task = [&]() {
        if (!reach(&task_full[nt % kTasks], (nt / kTasks) & 1u)) return false;
        it = tasks[nt % kTasks];
        return it.t0 < it.t1;
    };
    if (warp >= kProducer) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIo));
        if (warp == kProducer) {
            uint32_t kt = 0, vt = 0, items = 0;      // K tiles, V tiles and items under way or done
            bool ok = true;
            Walk walk;
            walk.plan(p);
            // 32 block ids, 8 tiles, at a time, one batch ahead; behind the end any block will do
            auto ids_from = [&](const Task &k, int t) {
                const int b = 4 * t + lane;
                return b < (k.L() + kBlock - 1) / kBlock ? p.block_tables[(int64_t)k.s * p.max_blocks_per_seq + b] : 0;
            };
            // the boxes of an item's query rows
            auto each_box = [&](const Task &k, auto &&box) {
                for (int i = 0; i < min(QT, k.n - k.first); i += p.box_tokens)
                    for (int rg = 0; rg < LY::kRegions; ++rg)
                        box(rg * kRows * 128 + i * G * 128, rg * 64, k.g, k.r0 + k.first + i);
            };
            Task after = walk.next(p);
            int ids_after = after.t0 < after.t1 ? ids_from(after, after.t0) : 0;
            for (;;) {
                it = after;
                if (nt >= kTasks)
                    ok = reach(&task_empty[nt % kTasks], (nt / kTasks - 1) & 1u);
                if (!ok) break;
                if (elect_one()) {
                    tasks[nt % kTasks] = it;
                    mbar_arrive(smem_addr(&task_full[nt % kTasks]));
                }
                ++nt;
                if (it.t0 >= it.t1) break;
                int ids = ids_after, ids_next = ids_from(it, it.t0 + 8);
                // the first row of the four blocks of tile t in the pools; all lanes call it
                auto rows_of = [&](int t, int (&y)[4]) {
                    bool bad = false;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        int id = __shfl_sync(kFull, ids, ((t - it.t0) & 7) * 4 + b);
                        if (id < 0 || id >= p.num_blocks) {
                            bad = true;
                            id = 0;
                        }
                        y[b] = (id * Hkv + it.g) * kBlock;
                    }
                    return bad;
                };
                auto copy = [&](const CUtensorMap *map, int at, uint64_t *bar, const int (&y)[4]) {
                    const uint32_t fb = smem_addr(bar), dst = smem_addr(smem + at);
                    mbar_arrive_expect_tx(fb, LY::kTileBytes);
#pragma unroll
                    for (int b = 0; b < 4; ++b)
#pragma unroll
                        for (int rg = 0; rg < LY::kRegions; ++rg)
                            tma_load_2d(dst + rg * kKeys * 128 + b * kBlock * 128, map, rg * 64, y[b], fb);
                };
                // K of a tile goes out before V of the tile before it
                int y_v[4] = {};
                for (int t = it.t0; t <= it.t1 && ok; ++t) {
                    int y[4] = {};
                    if (t < it.t1) {
                        if (((t - it.t0) & 7) == 0 && t > it.t0) {
                            ids = ids_next;
                            ids_next = ids_from(it, t + 8);
                        }
                        const bool bad = rows_of(t, y);
                        if (kt >= NK)
                            ok = reach(&k_empty[kt % NK], (kt / NK - 1) & 1u);
                        if (!ok) break;
                        if (elect_one()) {
                            if (bad) atomicOr(p.status, PKV_DEV_BAD_BLOCK);
                            bad_blocks[kt % kTilesKnown] = (uint8_t)bad;
                            copy(&tmK, LY::kKRing + (kt % NK) * LY::kTileBytes, &k_full[kt % NK], y);
                        }
                        ++kt;
                    }
                    if (t == it.t0) {
                        // the item's query rows, once its first K tile is under way
                        if (items > 0) ok = reach(q_empty, (items - 1) & 1u);
                        if (!ok) break;
                        ++items;
                        if (elect_one()) {
                            int boxes = 0;
                            each_box(it, [&](int, int, int, int) { ++boxes; });
                            const uint32_t qb = smem_addr(q_full);
                            mbar_arrive_expect_tx(qb, (uint32_t)(boxes * p.box_tokens * G * 128));
                            each_box(it, [&](int at, int x, int g, int token) {
                                tc::tma_load_4d(smem_addr(smem + at), &tmQ, x, 0, g, token, qb);
                            });
                        }
                    } else {
                        if (vt >= NV)
                            ok = reach(&v_empty[vt % NV], (vt / NV - 1) & 1u);
                        if (!ok) break;
                        if (elect_one())
                            copy(&tmV, LY::kVRing + (vt % NV) * LY::kTileBytes, &v_full[vt % NV], y_v);
                        ++vt;
                    }
#pragma unroll
                    for (int b = 0; b < 4; ++b) y_v[b] = y[b];
                    if (t == min(it.t0 + 1, it.t1)) {
                        // the item after this one: its first block ids, its query rows into L2
                        after = walk.next(p);
                        if (after.t0 < after.t1) {
                            ids_after = ids_from(after, after.t0);
                            if (elect_one())
                                each_box(after, [&](int, int x, int g, int token) {
                                    tc::tma_prefetch_4d(&tmQ, x, 0, g, token);
                                });
                        }
                    }
                }
                if (!ok) break;
            }
            // after a timed-out wait: let the copies still in flight land first
            if (*abort_flag && lane == 0) {
                auto drain = [&](uint64_t *bar, uint32_t parity) {
                    const unsigned long long t0 = globaltimer();
                    while (!mbar_try_wait(smem_addr(bar), parity))
                        if (globaltimer() - t0 > kTimeoutNs) break;
                };
                for (uint32_t i = kt > NK ? kt - NK : 0; i < kt; ++i) drain(&k_full[i % NK], (i / NK) & 1u);
                for (uint32_t i = vt > NV ? vt - NV : 0; i < vt; ++i) drain(&v_full[i % NV], (i / NV) & 1u);
                if (items > 0) drain(q_full, (items - 1) & 1u);
            }
        } else if (warp == kIssuer) {
            // bit 13 negates A: with a negative scale the products, so that all else counts up
            const uint32_t id_qk = tc::idesc_f16(BF16, kRows, kKeys, 0, 0) | (p.negate ? 1u << 13 : 0u);
            const uint32_t id_pv = tc::idesc_f16(BF16, kRows, D, 0, 1);
            const uint32_t t_s = __shfl_sync(kFull, tmem, 0), t_o = t_s + 128;
            const uint64_t qa_d = tc::desc_sw128(smem_addr(smem), 16, 1024);
            uint32_t kt = 0;                 // key tiles
            bool ok = true;
            // P V of tile vt
            auto issue_pv = [&](uint32_t vt) {
                const uint32_t slot = vt % NV, par = (vt / NV) & 1u, b = vt & 1u;
                ok = reach(&clean[slot], par) && reach(&v_full[slot], par) && reach(&p_full[b], (vt >> 1) & 1u);
                if (!ok) return;
                tc::fence_after_sync();
                const uint64_t vb_d =
                    tc::desc_sw128(smem_addr(smem + LY::kVRing + slot * LY::kTileBytes), kKeys * 128, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < 2 * kKeys / 16; ++i) {       // 16 keys, high or low parts
                        const int kk = 2 * (i >> 2) + (i & 1);
                        tc::mma_f16_ts(t_o, t_s + 64 * b + 8 * i, vb_d + (uint64_t)((kk * 16 * 128) >> 4),
                                       id_pv, true);
                    }
                    tc::mma_commit(smem_addr(&o_full[b]));
                    tc::mma_commit(smem_addr(&v_empty[slot]));
                }
                __syncwarp();
            };
            while (ok && next_task() && reach(q_full, nt & 1u)) {
#pragma unroll 1
                for (int t = it.t0; t <= it.t1; ++t) {
                    if (t < it.t1) {
                        const uint32_t slot = kt % NK;
                        if (!(ok = reach(&k_full[slot], (kt / NK) & 1u))) break;
                        tc::fence_after_sync();
                        const uint64_t kb_d =
                            tc::desc_sw128(smem_addr(smem + LY::kKRing + slot * LY::kTileBytes), 16, 1024);
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t off = (kk & 3) * 32;              // 16 values inside the row
                                tc::mma_f16(t_s + 64 * (kt & 1u),
                                            qa_d + (uint64_t)(((kk >> 2) * kRows * 128 + off) >> 4),
                                            kb_d + (uint64_t)(((kk >> 2) * kKeys * 128 + off) >> 4), id_qk, kk > 0);
                            }
                            tc::mma_commit(smem_addr(&s_full[kt & 1u]));
                            tc::mma_commit(smem_addr(&k_empty[slot]));
                            if (t == it.t1 - 1) tc::mma_commit(smem_addr(q_empty));
                        }
                        __syncwarp();
                    }
                    if (t > it.t0) issue_pv(kt - 1);
                    if (!ok) break;
                    if (t < it.t1) ++kt;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&task_empty[nt % kTasks]));
                ++nt;
            }
            // every MMA this warp issued has completed before the columns are freed
            if (elect_one()) {
                tc::mma_commit(smem_addr(done));
                const unsigned long long t0 = globaltimer();
                while (!mbar_try_wait(smem_addr(done), 0)) {
                    if (globaltimer() - t0 > kTimeoutNs) {
                        atomicOr(p.status, PKV_DEV_TIMEOUT);
                        break;
                    }
                }
            }
            __syncwarp();
        } else if (warp == kCleaner) {
            uint32_t vt = 0;
            bool ok = true;
            for (; ok && next_task(); ++nt) {
                for (int t = it.t0; t < it.t1; ++t, ++vt) {
                    const uint32_t slot = vt % NV;
                    if (!(ok = reach(&v_full[slot], (vt / NV) & 1u))) break;
                    const int k0 = t * kKeys;
                    if (k0 + kKeys > it.base) {
                        constexpr int kChunks = LY::kRegions * 8;
                        // chunk e of the tile's rows
                        auto chunk = [&](int e) -> uint4 & {
                            const int r = e / kChunks, c = e % kChunks;
                            return *reinterpret_cast<uint4 *>(smem + LY::kVRing + slot * LY::kTileBytes +
                                                              (c >> 3) * kKeys * 128 + r * 128 + (c & 7) * 16);
                        };
                        const int e0 = max(it.base - k0, 0) * kChunks, e1 = min(it.L() - k0, kKeys) * kChunks;
                        uint32_t sum[4] = {0u, 0u, 0u, 0u}, odd[2] = {0u, 0u};
#pragma unroll 2
                        for (int e = e0 + lane; e < e1; e += 32) {
                            const uint4 w = chunk(e);
                            add_odd<BF16>(sum[0], w.x);
                            add_odd<BF16>(sum[1], w.y);
                            add_odd<BF16>(sum[2], w.z);
                            add_odd<BF16>(sum[3], w.w);
                        }
#pragma unroll 1
                        for (int e = e1 + lane; e < kKeys * kChunks; e += 32) chunk(e) = make_uint4(0u, 0u, 0u, 0u);
                        if (__any_sync(kFull, odd_halves<BF16>(sum[0]) | odd_halves<BF16>(sum[1]) |
                                                  odd_halves<BF16>(sum[2]) | odd_halves<BF16>(sum[3]))) {
                            for (int e = e0 + lane; e < e1; e += 32) {
                                uint4 &w = chunk(e);
                                const uint4 o = make_uint4(odd_halves<BF16>(w.x), odd_halves<BF16>(w.y),
                                                           odd_halves<BF16>(w.z), odd_halves<BF16>(w.w));
                                if (o.x | o.y | o.z | o.w) {
                                    w = make_uint4(w.x & ~o.x, w.y & ~o.y, w.z & ~o.z, w.w & ~o.w);
                                    const int r = e / kChunks;
                                    odd[r >> 5] |= 1u << (r & 31);
                                }
                            }
                            odd[0] = __reduce_or_sync(kFull, odd[0]);
                            odd[1] = __reduce_or_sync(kFull, odd[1]);
                        }
                        if (lane == 0) odd_keys[slot] = odd[0] | (uint64_t)odd[1] << 32;
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive(smem_addr(&clean[slot]));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&task_empty[nt % kTasks]));
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---------------------------------------------------------- softmax
        const int r = threadIdx.x;
        const uint32_t t_s = tmem + ((uint32_t)(32 * warp) << 16), t_o = t_s + 128;
        const int jj = r / G, h = r - jj * G;
        uint32_t kt = 0;                 // key tiles
        bool alive = true;
        // the item is done with
        auto leave = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&task_empty[nt % kTasks]));
            ++nt;
        };
        while (alive && reach(&task_full[nt % kTasks], (nt / kTasks) & 1u)) {
            it = tasks[nt % kTasks];
            if (it.t0 >= it.t1) break;
            const int n = it.n, base = it.base, L = it.L();
            const int token = it.first + jj;
            const bool valid = r < QT * G && token < n;
            const bool busy = __any_sync(kFull, valid);  // some row of the warp counts
            const uint32_t *words = p.mask + (int64_t)(it.r0 + (valid ? token : it.first)) * p.words;
            const uint32_t w0 = words[0], w1 = p.words > 1 ? words[1] : 0u;
            float ref = kHide, l = 0.f;
            float sum_ref = kHide;                       // the reference of the moved sum, see kFlush
            int bad = 0;
            if (busy) {
                uint32_t z[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) z[c] = 0u;
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 32) tc::tmem_st32(t_o + c0, z);
            }
            for (int s0 = it.t0; alive && s0 < it.t1; s0 += kFlush) {
                const int s1 = min(s0 + kFlush, it.t1);
                for (int t = s0; t < s1; ++t, ++kt) {
                    const uint32_t b = kt & 1u, vslot = kt % NV;
                    if (!(alive = reach(&s_full[b], (kt >> 1) & 1u))) break;
                    if (!busy) {
                        if (lane == 0) mbar_arrive(smem_addr(&p_full[b]));
                        // (a barrier tells even phases from odd ones only: no phase is left out)
                        if (t > s0 && !(alive = reach(&o_full[b ^ 1u], ((kt - 1) >> 1) & 1u))) break;
                        continue;
                    }
                    tc::fence_after_sync();
                    bad |= bad_blocks[kt % kTilesKnown];
                    const int k0 = t * kKeys;
                    const bool edge = k0 + kKeys > base;     // drafted tokens or the end: masks
                    uint64_t see = ~0ull;
                    if (edge && valid) see = seen_keys(p, words, w0, w1, k0, base, L);
                    // the tile's products (the scale is in the exponents), those that the row does not see
                    // hidden; read once (twice, 32 at a time: 22 sequences of 25,000 tokens in 3 heads
                    // of 64 take 93 us in place of 85)
                    float x[kKeys];
                    {
                        uint32_t v[2][32];
                        tc::tmem_ld32(t_s + 64 * b, v[0]);
                        tc::tmem_ld32(t_s + 64 * b + 32, v[1]);
                        tc::tmem_wait_ld();
    #pragma unroll
                        for (int c = 0; c < kKeys; ++c) x[c] = __uint_as_float(v[c / 32][c % 32]);
                    }
                    if (edge) {
    #pragma unroll
                        for (int c = 0; c < kKeys; ++c)
                            if (!((uint32_t)(see >> (c & 32)) >> (c & 31) & 1u)) x[c] = kHide;
                    }
                    // the largest, in four chains (one of 32 steps would be waited for)
                    float m[4] = {kHide, kHide, kHide, kHide};
    #pragma unroll
                    for (int c = 0; c < kKeys; c += 2) m[c / 2 % 4] = max3f(m[c / 2 % 4], x[c], x[c + 1]);
                    const float mx = fmaxf(max3f(m[0], m[1], m[2]), m[3]);
                    // The reference is a product: a weight is 2^((x - ref) scale + kTop), so products
                    // that agree weigh alike whatever their size, and nothing is lost to the rounding
                    // of a scaled reference.
                    float f = 1.f;
                    bool resc = false;
                    const bool unset = ref == kHide;          // no key seen yet
                    if (valid && mx != kHide && (unset || (mx - ref) * p.scale_log2 > kLazy)) {
                        if (!unset) {
                            f = fast_exp2((ref - mx) * p.scale_log2);
                            resc = true;
                        }
                        ref = mx;
                    }
                    // (any finite reference gives hidden products weight 2^-inf = 0)
                    const float sub = ref == kHide ? 0.f : ref;
                    const uint64_t sc2 = pack2f(p.scale_log2, p.scale_log2), sub2 = pack2f(-sub, -sub);
                    const uint64_t top2 = pack2f(kTop, kTop);
                    uint64_t lsum2 = pack2f(0.f, 0.f);
                    // weights over the products' columns: 16 of high parts, 16 of low parts
    #pragma unroll
                    for (int c0 = 0; c0 < kKeys; c0 += 32) {
                        uint32_t hi[16], lo[16];
    #pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            const uint64_t d2 = add2f(pack2f(x[c0 + c], x[c0 + c + 1]), sub2);
                            const float2 e = unpack2f(kTop == 0.f ? mul2f(d2, sc2) : fma2f(d2, sc2, top2));
                            const float p0 = fast_exp2(e.x), p1 = fast_exp2(e.y);
                            const uint64_t pp = pack2f(p0, p1);
                            lsum2 = add2f(lsum2, pp);
                            two_parts<BF16>(p0, p1, pp, hi[c / 2], lo[c / 2]);
                        }
                        tc::tmem_st16(t_s + 64 * b + c0, hi);
                        tc::tmem_st16(t_s + 64 * b + c0 + 16, lo);
                    }
                    const float2 ls = unpack2f(lsum2);
                    l = l * f + (ls.x + ls.y);
                    uint64_t odd = 0ull;                     // keys whose V held odd values
                    if (edge) {
                        if (!(alive = reach(&clean[vslot], (kt / NV) & 1u))) break;
                        odd = odd_keys[vslot];
                    }
                    // O changes before P V of this tile, once P V of the one before has ended; the
                    // wait for that consumes its o_full phase either here or after P is out
                    const bool touch = __any_sync(kFull, resc) || odd;
                    if (touch && t > s0) {
                        if (!(alive = reach(&o_full[b ^ 1u], ((kt - 1) >> 1) & 1u))) break;
                        tc::fence_after_sync();
                    }
                    if (touch) {
                        tc::tmem_wait_st();                  // (O's zeros, in an item's first tile; P)
    #pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t v[32];
                            tc::tmem_ld32(t_o + c0, v);
                            tc::tmem_wait_ld();
    #pragma unroll
                            for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * f);
                            tc::tmem_st32(t_o + c0, v);
                        }
                        tc::tmem_wait_st();
                        // the odd values of a key's V go to the rows that see it, times their weights
                        // (an infinity, or NaN; 0 * infinity is NaN)
    #pragma unroll 1
                        for (uint64_t left = odd; left; left &= left - 1) {
                            const int c = __ffsll((long long)left) - 1, pos = k0 + c;
                            const uint32_t word = t_s + 64 * b + (c & 32) + (c & 31) / 2;
                            const uint32_t both = column(word) | column(word + 16);
                            const bool some = (both >> (16 * (c & 1)) & 0x7fffu) != 0u;
                            int id = p.block_tables[(int64_t)it.s * p.max_blocks_per_seq + pos / kBlock];
                            if (id < 0 || id >= p.num_blocks) id = 0;            // (the result is zero anyway)
                            const T *vp = static_cast<const T *>(p.v_pool) +
                                          (((int64_t)id * Hkv + it.g) * kBlock + pos % kBlock) * D;
    #pragma unroll 1
                            for (int d = 0; d < D; ++d) {
                                const float y = (float)vp[d];
                                if (fabsf(y) < INFINITY) continue;               // the same for the warp
                                const float o = __uint_as_float(column(t_o + d));
                                set_column(t_o + d, __float_as_uint(see >> c & 1u ? o + (some ? y : NAN) : o));
                            }
                        }
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&p_full[b]));
                    if (!touch && t > s0) {
                        if (!(alive = reach(&o_full[b ^ 1u], ((kt - 1) >> 1) & 1u))) break;
                    }
                }
                if (!alive) break;
                // the last P V is done (which writes the lanes of warps without rows too: they wait before
                // another item's zeros)
                if (!(alive = reach(&o_full[(kt - 1) & 1u], ((kt - 1) >> 1) & 1u))) break;
                tc::fence_after_sync();
                if (busy && it.t1 - it.t0 > kFlush) {
                    move_sum<D>(p, t_o, it.t0 == 0, valid, s0 > it.t0, sum_ref, ref, s1 == it.t1);
                    sum_ref = ref;
                }
            }
            if (!alive) break;
            // ---- the part's result
            if (!busy) {
                leave();
                continue;
            }
            if (it.t0 > 0 || it.t1 * kKeys < L) {
                const int64_t piece = 2 * blockIdx.x + (it.t0 == 0);
                if (valid) p.part_ml[piece * p.piece_rows + r] = make_float2(ref, bad ? -1.f : l);
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t v[32];
                    tc::tmem_ld32(t_o + c0, v);
                    tc::tmem_wait_ld();
                    if (valid) {
                        float4 *dst = p.part_o + (piece * (D / 4) + c0 / 4) * p.piece_rows + r;
#pragma unroll
                        for (int c = 0; c < 32; c += 4)
                            dst[(int64_t)(c / 4) * p.piece_rows] =
                                make_float4(__uint_as_float(v[c]), __uint_as_float(v[c + 1]),
                                            __uint_as_float(v[c + 2]), __uint_as_float(v[c + 3]));
                    }
                }
            } else {
                const bool none = bad || l == 0.f;       // a bad block, or nothing seen
                const float inv = none ? 0.f : 1.f / l;
                T *out = static_cast<T *>(p.out) +
                         ((int64_t)(it.r0 + token) * p.num_q_heads + (int64_t)it.g * G + h) * D;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t v[32];
                    tc::tmem_ld32(t_o + c0, v);
                    tc::tmem_wait_ld();
                    if (valid) {
#pragma unroll
                        for (int c = 0; c < 32; c += 8) {
                            auto two_of = [&](int k) {
                                return none ? 0u : E::pack(__uint_as_float(v[c + k]) * inv,
                                                           __uint_as_float(v[c + k + 1]) * inv);
                            };
                            *reinterpret_cast<uint4 *>(out + c0 + c) =
                                make_uint4(two_of(0), two_of(2), two_of(4), two_of(6));
                        }
                    }
                }
            }
            tc::fence_before_sync();
            leave();
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, kColumns);
}

// ------------------------------------------------------------------ joining the pieces
// A task is 32 rows and 8 columns of a cut item; one, two, four or eight warps share its pieces
// (in turn, so that the order of a sum does not vary), four pieces under way at a time, and
// meet in shared memory.  Every CTA lists the cut items and their passes (as many tasks as a CTA
// takes at once), and takes every gridDim-th pass.  A CTA to an SM: 4 sequences 22.4 us (27 with
// half as many, 23 with twice).
constexpr int kJoinThreads = 512, kJoinWarps = kJoinThreads / 32, kJoinCtas = 152;
static_assert(kJoinThreads >= kMaxRanges, "a thread for each range");

__device__ __forceinline__ int ways_of(int pieces) { return pieces > 16 ? 8 : pieces > 8 ? 4 : pieces > 4 ? 2 : 1; }

__device__ __forceinline__ int tasks_of(const Params &p, int D, int tokens)
{
    return (tokens * p.group + 31) / 32 * (D / 8);
}

// Zero rows for the sequences whose lengths do not fit: their number of rows is whatever the
// caller gave, so all CTAs share them (in the main kernel others would wait for the CTA that
// does it).
template <int D>
__device__ __noinline__ void clear_refused(const Params &p)
{
    const int lane = threadIdx.x & 31;
    for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
        const int i = min(s0 + lane, p.num_seqs - 1);
        const Seq x = seq_of(p, p.query_start[i], p.query_start[i + 1], p.context_lens[i]);
        for (unsigned bad = __ballot_sync(kFull, s0 + lane < p.num_seqs && x.bad); bad; bad &= bad - 1) {
            const int src = __ffs(bad) - 1;
            const int64_t row = (int64_t)p.num_q_heads * (D / 8);        // in 16-byte chunks
            const int64_t all = row * __shfl_sync(kFull, x.n, src);
            uint4 *out = static_cast<uint4 *>(p.out) + row * (all ? __shfl_sync(kFull, x.r0, src) : 0);
            for (int64_t c = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; c < all;
                 c += (int64_t)gridDim.x * kJoinThreads)
                out[c] = make_uint4(0, 0, 0, 0);
        }
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads, 1) tree_join_kernel(const Params p)
{
    using E = Elem<BF16>;
    using T = typename E::T;
    __shared__ int4 ranges[kMaxRanges];
    __shared__ int begins[kMaxRanges], ends[kMaxRanges], passes[kMaxRanges + 1], sums[kJoinWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_launch_dependents();
    griddep_wait();
    // the sum of the warps' totals before this one, and of all
    auto across = [&](int total, int &all) {
        if (lane == 0) sums[warp] = total;
        __syncthreads();
        const int x = lane < kJoinWarps ? sums[lane] : 0;
        all = __reduce_add_sync(kFull, x);
        return (int)__reduce_add_sync(kFull, lane < warp ? x : 0);
    };
    int4 range = make_int4(0, 0, 0, 0);
    if (tid < p.grid) ranges[tid] = range = p.ranges[tid];
    if (p.ranges[0].x & kRefused) clear_refused<D>(p);
    const unsigned begun = __ballot_sync(kFull, range.x & kBegins);
    int items;
    const int rank = across(__popc(begun), items) + __popc(begun & ((1u << lane) - 1u));
    if (range.x & kBegins) begins[rank] = tid;
    if (range.x & kEnds) ends[rank - 1] = tid;           // the item begun before this range's own
    __syncthreads();
    int n = 0;
    if (tid < items) {
        const int per_pass = kJoinWarps / ways_of(ends[tid] - begins[tid] + 1);
        n = (tasks_of(p, D, ranges[begins[tid]].y) + per_pass - 1) / per_pass;
    }
    int upto = n, all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += y;
    }
    upto += across(__shfl_sync(kFull, upto, 31), all);
    if (tid < items) passes[tid] = upto - n;
    if (tid == 0) passes[items] = all;
    __syncthreads();
    const int G = p.group;
    const float sc = p.scale_log2;
    __shared__ float shares[kJoinWarps][11][32];
    for (int pass = blockIdx.x; pass < passes[items]; pass += gridDim.x) {
        int item = 0;                                    // the last item that begins at or before the pass
        for (int step = 256; step > 0; step >>= 1)
            if (item + step < items && passes[item + step] <= pass) item += step;
        const int begin = begins[item], pieces = ends[item] - begin + 1;
        const int tokens = ranges[begin].y, row0 = ranges[begin].z, g = ranges[begin].w;
        const int tasks = tasks_of(p, D, tokens), ways = ways_of(pieces), mine = warp % ways;
        const int task = (pass - passes[item]) * (kJoinWarps / ways) + warp / ways;
        const int rr = task / (D / 8) * 32 + lane, c8 = task % (D / 8);
        const int token = rr / G, h = rr - token * G;
        const bool valid = task < tasks && token < tokens;
        float ref = kHide, l = 0.f, o[8] = {};
        bool bad = false;
        auto add = [&](float2 ml, const float (&v)[8]) {
            bad |= ml.y < 0.f;
            if (ml.y == 0.f) return;                     // nothing seen there
            const float now = fmaxf(ref, ml.x);
            const float f = ref == kHide ? 0.f : fast_exp2((ref - now) * sc);
            const float w = fast_exp2((ml.x - now) * sc);
            ref = now;
            l = l * f + w * ml.y;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = o[e] * f + w * v[e];
        };
        const float2 *ml_at = p.part_ml + rr;
        const float4 *o_at = p.part_o + (int64_t)2 * c8 * p.piece_rows + rr;
        for (int k0 = mine; k0 < pieces && valid; k0 += 4 * ways) {
            float2 ml[4];
            float4 a[4], b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = k0 + k * ways;
                if (at >= pieces) break;
                const int64_t piece = at == 0 ? 2 * begin + 1 : 2 * (begin + at);
                const float4 *src = o_at + piece * (D / 4) * p.piece_rows;
                ml[k] = ml_at[piece * p.piece_rows];
                a[k] = src[0];
                b[k] = src[p.piece_rows];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k0 + k * ways < pieces)
                    add(ml[k], {a[k].x, a[k].y, a[k].z, a[k].w, b[k].x, b[k].y, b[k].z, b[k].w});
        }
        if (ways > 1) {                                  // the same for the CTA
            float (&share)[11][32] = shares[warp];
            if (mine) {
                share[0][lane] = ref;
                share[1][lane] = l;
                share[2][lane] = bad ? 1.f : 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) share[3 + e][lane] = o[e];
            }
            __syncthreads();
            if (mine == 0) {
                for (int w = 1; w < ways; ++w) {
                    const float (&other)[11][32] = shares[warp + w];
                    bad |= other[2][lane] != 0.f;
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = other[3 + e][lane];
                    // (its output is in terms of its own reference and sum)
                    add(make_float2(other[0][lane], other[1][lane]), v);
                }
            }
            __syncthreads();
        }
        if (!valid || mine) continue;
        const bool none = bad || l == 0.f;
        const float inv = none ? 0.f : 1.f / l;
        auto two_of = [&](int k) { return none ? 0u : E::pack(o[k] * inv, o[k + 1] * inv); };
        T *out = static_cast<T *>(p.out) +
                 ((int64_t)(row0 + token) * p.num_q_heads + (int64_t)g * G + h) * D + 8 * c8;
        *reinterpret_cast<uint4 *>(out) = make_uint4(two_of(0), two_of(2), two_of(4), two_of(6));
    }
}

// --------------------------------------------------------------------- host side
using EncodeFn = PFN_cuTensorMapEncodeTiled_v12000;

static EncodeFn encode_fn()
{
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(ptr);
    });
    return fn;
}

static bool make_map(CUtensorMap *map, const void *base, bool bf16, int rank, const cuuint64_t *dims,
                     const cuuint64_t *strides, const cuuint32_t *box)
{
    const EncodeFn enc = encode_fn();
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return enc && enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                      (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, step,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tokens of a box of query rows: whole groups of 8 rows (the swizzle's atom), about 32 rows.
static int box_tokens(int G)
{
    const int unit = G % 8 == 0 ? 1 : G % 4 == 0 ? 2 : G % 2 == 0 ? 4 : 8;
    return unit * std::max(1, 32 / (unit * G));
}

static int tile_tokens(int G) { return kRows / (box_tokens(G) * G) * box_tokens(G); }

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Rows of a piece's place: a call whose rows fit less than a query tile needs less.
static int64_t piece_rows(int64_t T, int G) { return std::min<int64_t>(kRows, (T * G + 31) / 32 * 32); }

struct Workspace {
    size_t ranges, ml, o, total;
};
static Workspace workspace_of(int64_t T, int G, int D)
{
    const size_t rows = 2 * kMaxRanges * (size_t)piece_rows(T, G);
    Workspace w;
    w.ranges = 0;
    w.ml = w.ranges + align256(kMaxRanges * sizeof(int4));
    w.o = w.ml + align256(rows * sizeof(float2));
    w.total = w.o + rows * D * sizeof(float);
    return w;
}

using KernelFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, Params);
using JoinFn = void (*)(Params);

struct Pick {
    KernelFn fn;
    JoinFn join;
    int smem;
};

template <int D, bool BF16>
static Pick pick_of()
{
    return {&tree_kernel<D, BF16>, &tree_join_kernel<D, BF16>, Layout<D>::kTotal};
}

// CTAs of a kernel that fit the current device at once, cached per device and kernel.  (The
// runtime's own count is one to an SM for every kernel that allocates tensor memory; two of
// these take 512 columns, all there are.)
static int resident(const Pick &k, int slot)
{
    constexpr int kMaxDev = 64, kSlots = 4;
    static std::mutex mu;
    static int ctas[kMaxDev][kSlots];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return -1;
    std::lock_guard<std::mutex> lock(mu);
    int &n = ctas[dev][slot];
    if (n == 0) {
        const void *fn = reinterpret_cast<const void *>(k.fn);
        int sms = 0, shared = 0, reserved = 0;
        cudaFuncAttributes a;
        if (cudaFuncGetAttributes(&a, fn) != cudaSuccess || a.numRegs != kLaunchRegs) return -1;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&shared, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev) != cudaSuccess ||
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem) != cudaSuccess ||
            cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared) != cudaSuccess)
            return -1;
        n = sms * (2 * (k.smem + reserved) <= shared ? 2 : 1);
    }
    return n;
}

}  // namespace tree
}  // namespace pkv

extern "C" size_t paged_tree_workspace_bytes(int32_t num_tokens, int32_t num_q_heads,
                                             int32_t num_kv_heads, int32_t head_dim)
{
    if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
        num_q_heads / num_kv_heads > 16 || (head_dim != 64 && head_dim != 128))
        return 0;
    return pkv::tree::workspace_of(num_tokens, num_q_heads / num_kv_heads, head_dim).total;
}

extern "C" int paged_tree_attention(const pkv_pool *pool, void *out, const void *q,
                                    const void *k_pool, const void *v_pool,
                                    const int32_t *block_tables, int32_t max_blocks_per_seq,
                                    const int32_t *query_start, const int32_t *context_lens,
                                    const int32_t *tree_mask, int32_t mask_words, int32_t num_seqs,
                                    int32_t num_tokens, int32_t num_q_heads, float scale,
                                    void *workspace, size_t workspace_bytes, int32_t *d_status,
                                    void *stream)
{
    using namespace pkv::tree;
    pkv::PoolGeometry g;
    if (!pkv::pool_geometry(pool, &g) || !pkv::is_16bit(g)) return PKV_ERR_INVALID_ARG;
    if (num_seqs < 0 || num_tokens < 0 || num_q_heads <= 0 || max_blocks_per_seq <= 0 ||
        mask_words < 1 || mask_words > kMaxWords || num_q_heads % g.num_kv_heads)
        return PKV_ERR_INVALID_ARG;
    if (!(scale == scale) || scale == INFINITY || scale == -INFINITY) return PKV_ERR_INVALID_ARG;
    const int G = num_q_heads / g.num_kv_heads, D = g.head_dim;
    if (g.block_size != pkv::kBlock || G > 16 || (D != 64 && D != 128)) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !query_start || !context_lens ||
        !tree_mask || !workspace || !d_status)
        return PKV_ERR_INVALID_ARG;
    if (!pkv::aligned16(out) || !pkv::aligned16(q) || !pkv::aligned16(k_pool) ||
        !pkv::aligned16(v_pool) || ((uintptr_t)workspace & 255u) ||
        ((uintptr_t)block_tables & 3u) || ((uintptr_t)query_start & 3u) ||
        ((uintptr_t)context_lens & 3u) || ((uintptr_t)tree_mask & 3u) || ((uintptr_t)d_status & 3u))
        return PKV_ERR_INVALID_ARG;
    const Workspace ws = workspace_of(num_tokens, G, D);
    if (workspace_bytes < ws.total) return PKV_ERR_INVALID_ARG;
    if ((int64_t)g.num_blocks * g.num_kv_heads * g.block_size > (int64_t)1 << 31)
        return PKV_ERR_UNSUPPORTED;
    const bool bf16 = g.dtype == PKV_BF16;
    const Pick k = D == 128 ? (bf16 ? pick_of<128, true>() : pick_of<128, false>())
                            : (bf16 ? pick_of<64, true>() : pick_of<64, false>());

    Params prm;
    prm.out = out;
    prm.v_pool = v_pool;
    prm.block_tables = block_tables;
    prm.query_start = query_start;
    prm.context_lens = context_lens;
    prm.mask = reinterpret_cast<const uint32_t *>(tree_mask);
    prm.words = mask_words;
    prm.num_seqs = num_seqs;
    prm.num_tokens = num_tokens;
    prm.num_q_heads = num_q_heads;
    prm.num_kv_heads = g.num_kv_heads;
    prm.group = G;
    prm.max_blocks_per_seq = max_blocks_per_seq;
    prm.max_tokens = (int32_t)std::min<int64_t>((int64_t)max_blocks_per_seq * pkv::kBlock,
                                                 INT32_MAX - 2 * kKeys);
    prm.num_blocks = g.num_blocks;
    prm.tile_tokens = tile_tokens(G);
    prm.box_tokens = box_tokens(G);
    prm.tile_inverse = ((1 << 20) + prm.tile_tokens - 1) / prm.tile_tokens;
    prm.piece_rows = (int32_t)piece_rows(num_tokens, G);
    // the ranges are counted in 32 bits, whatever the row ranges hold
    const int64_t tiles_of_seq = (std::min(num_tokens, 32 * mask_words) + prm.tile_tokens - 1) / prm.tile_tokens;
    const double most = (double)num_seqs * tiles_of_seq * g.num_kv_heads * (prm.max_tokens / kKeys + 1 + kItemCost);
    if (most > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    // Scores are hidden by an infinity that the scale must carry into the exponent, and a product
    // that is the reference must weigh 1: the scale is a finite normal number.  At scale 0 the
    // smallest one weighs all keys alike.
    prm.scale_log2 = std::min(std::max(fabsf(scale) * 1.4426950408889634f, FLT_MIN), FLT_MAX);
    prm.negate = scale < 0.f;
    char *w = static_cast<char *>(workspace);
    prm.ranges = reinterpret_cast<int4 *>(w + ws.ranges);
    prm.part_ml = reinterpret_cast<float2 *>(w + ws.ml);
    prm.part_o = reinterpret_cast<float4 *>(w + ws.o);
    prm.status = d_status;

    CUtensorMap tk, tv, tq;
    const cuuint64_t rows[2] = {(cuuint64_t)D, (cuuint64_t)g.num_blocks * g.num_kv_heads * g.block_size};
    const cuuint64_t row_bytes[1] = {(cuuint64_t)D * 2};
    const cuuint32_t block[2] = {64u, (cuuint32_t)pkv::kBlock};
    // query rows as (D, G, Hkv, T): a box brings G rows of each of its tokens
    const cuuint64_t qd[4] = {(cuuint64_t)D, (cuuint64_t)G, (cuuint64_t)g.num_kv_heads, (cuuint64_t)num_tokens};
    const cuuint64_t qs[3] = {(cuuint64_t)D * 2, (cuuint64_t)G * D * 2, (cuuint64_t)num_q_heads * D * 2};
    const cuuint32_t qb[4] = {64u, (cuuint32_t)G, 1u, (cuuint32_t)prm.box_tokens};
    if (!make_map(&tk, k_pool, bf16, 2, rows, row_bytes, block) ||
        !make_map(&tv, v_pool, bf16, 2, rows, row_bytes, block) || !make_map(&tq, q, bf16, 4, qd, qs, qb))
        return PKV_ERR_CUDA;
    const int fit = resident(k, (D == 128) * 2 + bf16);
    if (fit < 1) return PKV_ERR_CUDA;

    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    // no more CTAs than the tables' rows hold units (one small tree 10.1 -> 9.7 us)
    prm.grid = (int)std::min<double>(std::min(fit, kMaxRanges), std::max(1.0, most));
    cfg.gridDim = dim3((unsigned)prm.grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)k.smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k.fn, tk, tv, tq, prm) != cudaSuccess) return PKV_ERR_CUDA;
    cfg.gridDim = dim3(kJoinCtas);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, k.join, prm) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
