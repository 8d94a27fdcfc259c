// Single-token attention over the visible part of each sequence's cache: the
// last `window` tokens and the first `sinks` tokens, over a 16-bit pool or a
// block-scaled 8-bit pool (there also over the whole context).
//
//   x_j = scale <q, K_j>,  out = sum_j softmax(x)_j V_j   over the visible j:
//   j < L  and  (j >= L - window  or  j < sinks)
//
// One launch, no workspace.  A (sequence, kv head) pair is one cluster of C CTAs
// (C = 1: a plain CTA).  Its visible blocks -- the sinks' blocks, then the
// window's, numbered without the gap between them -- are dealt to the cluster's
// warps in turn.  Each warp is its own producer: it keeps a private ring of
// stages, lane 0 copies block i + kStages (TMA) as soon as block i is consumed,
// and block ids are fetched 32 at a time, one batch ahead.  The warps' (o, max,
// sum) meet in shared memory, the CTAs' through distributed shared memory, always
// in the same order, so results do not vary from run to run.  Where the grid is
// more than one wave of ragged lengths, the longest pairs go first.
//
// Per 16-token block and warp, everything on mma.sync m16n8k16 with the tokens
// (then the dimensions) as the 16 rows and eight query heads as the columns:
//   S^T = K Q^T        rows = tokens, columns = heads
//   P   = 2^(S - m)    fp32, against a lazy reference maximum m
//   O^T += V^T P^T     rows = dimensions; P^T comes from S^T's accumulator
//                      layout through one 8x8 transpose (movmatrix) per half
// so no half of a matrix instruction works on empty rows (G <= 8), and the
// statistics and the accumulators of a head sit in the same lanes.  (tcgen05
// takes 64 or 128 rows: with G <= 16 query rows per pair and a new K tile each
// step it would idle; the tensor pipe is 18 to 28 % busy here.)
//
// The bytes of the visible K and V bound it, each read once: 256 sequences x 8
// kv heads x window 1,024 (16-bit, 1.05 GB) 155 us, 6.8 TB/s; 160 ragged contexts
// of up to 16,384 tokens (8-bit, 2.87 GB) 422 us, 6.8 TB/s.  Where a few pairs
// leave SMs idle, an SM's own pace counts: 46 GB/s of 8-bit blocks (360
// instructions per block and warp, half of the issue slots; 57 GB/s and 280 with
// weights in one part and codes that kept their offset, see consume_b8).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "decode_params.h"
#include "pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace window {

constexpr int kMaxHeads = 16;            // query heads per kv head
// The reference maximum moves only when a score exceeds it by more than kLazy (log2
// units).  Where weights become fp16 (fp16 and 8-bit pools) it is taken kTop below the
// largest score: weights stay within 2^14, the largest is at least 2^8, and those down
// to 2^-22 of it are normal numbers in fp16 (2^-14 with the reference at the maximum: a
// long context far below a few dominant tokens would lose its weights' bits).
constexpr float kLazy = 6.f, kTop = 8.f, kTopInverse = 0x1p-8f;

struct Params {
    void *out;
    const void *q;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const uint8_t *kv;                   // 8-bit records
    int32_t num_q_heads, num_kv_heads, group, max_blocks_per_seq, num_blocks;
    int32_t window, sinks;               // window >= 1 (INT32_MAX: all)
    int32_t ctas;                        // cluster size C
    float scale_log2;
    int32_t *status;
    int32_t num_seqs;
    int32_t most;                        // > 0: pairs run longest first; the most blocks one can show
};

using KernelFn = void (*)(CUtensorMap, CUtensorMap, Params);

// Visible blocks of a sequence of L tokens: logical blocks 0 .. sink_blocks - 1
// and those from sink_blocks + gap on; n in all.
struct Visible {
    int L, lo, sinks, sink_blocks, gap, n;
    __device__ __forceinline__ int block(int v) const { return v < sink_blocks ? v : v + gap; }
    // some token of logical block b is hidden
    __device__ __forceinline__ bool partial(int b) const
    {
        const int t0 = b * kBlock;
        return t0 + kBlock > L || (t0 < lo && t0 + kBlock > sinks);
    }
    // bit t: token t of logical block b is visible
    __device__ __forceinline__ uint32_t mask(int b) const
    {
        auto below = [](int x) { return x <= 0 ? 0u : x >= kBlock ? 0xffffu : (1u << x) - 1u; };
        const int t0 = b * kBlock;
        return below(L - t0) & (~below(lo - t0) | below(sinks - t0));
    }
};

__device__ __forceinline__ Visible visible(int L, int window, int sinks)
{
    Visible v;
    v.L = L;
    v.lo = max(0, L - window);
    v.sinks = min(sinks, L);
    v.sink_blocks = (v.sinks + kBlock - 1) / kBlock;
    v.gap = max(0, v.lo / kBlock - v.sink_blocks);
    v.n = (L + kBlock - 1) / kBlock - v.gap;
    return v;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Shared-memory address `addr` of this CTA in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}

__device__ __forceinline__ float4 cluster_load4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float2 cluster_load2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr)
                 : "memory");
    return v;
}

// Shapes of one variant.  B8: block-scaled 8-bit records; else 16-bit pools.
template <int D, bool B8, int NT, int W>
struct Shape {
    static constexpr int kThreads = 32 * W;
    static constexpr int kCopyBytes = B8 ? 32 * D + 16 : 64 * D;       // of one block and head
    static constexpr int kStageBytes = B8 ? (32 * D + 16 + 127) / 128 * 128 : 64 * D;
    // stages per warp: 16-bit 24 KB in flight, 2 CTAs per SM; 8-bit 16 KB, 3 CTAs per SM
    static constexpr int kStages = B8 ? (D == 128 ? 4 : 8) : (D == 128 ? 3 : 6);
    static constexpr int kMinBlocks = W > 4 ? 1 : B8 && NT == 1 ? 3 : 2;
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kRow = D + 4;                                  // floats of a merge row
    static constexpr int kBars = W * kWarpBytes;
    static constexpr int kMl = kBars + W * 8 * 8;                       // [warps + 1][16] float2
    static constexpr int kTotal = 1024 + kMl + (W + 1) * kMaxHeads * 8;
    static_assert(kStages <= 8 && 8 * NT * kRow * 4 <= kWarpBytes, "merge rows fit a warp's ring");
};

// A warp's running state for NT tiles of eight heads: lane (r, q4) = (lane / 4,
// lane % 4) holds heads 2 q4 and 2 q4 + 1 of each tile; o[nt][m] = (dimension
// A, head 0), (A, head 1), (B, head 0), (B, head 1) of 16-dimension tile m.
template <int D, int NT>
struct State {
    float o[NT][D / 16][4];
    // reference maximum m = -neg; 0 and bit 2 nt + h of `unset` before a head's first
    // finite score (m = -inf)
    float neg[NT][2], l[NT][2];
    uint32_t unset;
    bool special;                        // some head of the warp is unset or has |m| > 2^24
    __device__ __forceinline__ float m(int nt, int h) const
    {
        return (unset >> (2 * nt + h)) & 1u ? -INFINITY : -neg[nt][h];
    }
};

// The query rows of a kv head as B operands (head r of tile nt); for 8-bit pools
// also each row's scale, for heads 2 q4 and 2 q4 + 1.
template <int D, int NT>
struct Queries {
    uint32_t b[NT][D / 16][2];
    float scale[NT][2];
};

template <int D, int NT>
__device__ __forceinline__ void reset(State<D, NT> &st)
{
    st.unset = ~0u;
    st.special = true;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        st.neg[nt][0] = st.neg[nt][1] = 0.f;
        st.l[nt][0] = st.l[nt][1] = 0.f;
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.o[nt][t][e] = 0.f;
    }
}

// Products x of tokens r and r + 8 of NB blocks -> weights 2^(x f - m), with the
// lazy reference maximum m; x[b][nt] = (r, head 0), (r, head 1), (r + 8, head 0),
// (r + 8, head 1), f[b][nt] = the heads' factors to the log2 domain, hidden
// tokens' bits 0 in masks[b].
// A weight depends on its product and on m alone, whatever the block and the path by
// which m came about: the exponent is taken from the product itself (one fma, the
// product not rounded), also when this block moves m, and what was summed before is
// scaled by the exact step of m.  Products beyond 2^24, whose spacing is a unit and
// more, are rounded like the maximum that m was taken from (`wide`): unrounded ones
// would lie up to half that spacing above it.  top = kTop where weights become fp16, else 0.
template <int D, int NT, int NB>
__device__ __forceinline__ void softmax_step(State<D, NT> &st, float (&x)[NB][NT][4],
                                             const float (&f)[NB][NT][2], const uint32_t (&masks)[NB],
                                             float top, int lane)
{
    float y[NB][NT][4];                  // exponents, -inf for hidden tokens
    auto hide = [&]() {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (masks[b] == 0xffffu) continue;           // the same for the warp
            const bool v0 = (masks[b] >> (lane >> 2)) & 1u, v1 = (masks[b] >> ((lane >> 2) + 8)) & 1u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!(e < 2 ? v0 : v1)) y[b][nt][e] = -INFINITY;
        }
    };
    auto each = [&](auto exponent) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[b][nt][e] = exponent(x[b][nt][e], f[b][nt][e & 1], nt, e & 1);
        hide();
    };
    each([&](float p, float factor, int nt, int h) { return fmaf(p, factor, st.neg[nt][h]); });
    bool raise = st.special;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) raise |= y[b][nt][e] > top + kLazy;
    if (__any_sync(kFull, raise)) {      // m moves, or the warp is special: products of their own
        each([&](float p, float factor, int, int) { return __fmul_rn(p, factor); });
        auto is_wide = [](float m) { return m != -INFINITY && fabsf(m) > 0x1p24f; };
        bool special = false;
        uint32_t wide = 0u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float up = fmaxf(y[0][nt][h], y[0][nt][2 + h]);
#pragma unroll
                for (int b = 1; b < NB; ++b) up = fmaxf(up, fmaxf(y[b][nt][h], y[b][nt][2 + h]));
                up = fmaxf(up, __shfl_xor_sync(kFull, up, 4));
                up = fmaxf(up, __shfl_xor_sync(kFull, up, 8));
                up = fmaxf(up, __shfl_xor_sync(kFull, up, 16));
                // the reference moves up with the largest score (from 2^24 on, where
                // the spacing nears kTop, to it)
                const float old = st.m(nt, h);
                const float now = fmaxf(old, fabsf(up) > 0x1p24f ? up : up - top);
                const float s = old == -INFINITY ? 1.f : fast_exp2(old - now);
                if (now != -INFINITY) {
                    st.neg[nt][h] = -now;
                    st.unset &= ~(1u << (2 * nt + h));
                }
                if (is_wide(now)) wide |= 1u << (2 * nt + h);
                special |= now == -INFINITY || is_wide(now);
                st.l[nt][h] *= s;
#pragma unroll
                for (int t = 0; t < D / 16; ++t) {
                    st.o[nt][t][h] *= s;
                    st.o[nt][t][2 + h] *= s;
                }
            }
        }
        st.special = __any_sync(kFull, special);
        each([&](float p, float factor, int nt, int h) {
            return (wide >> (2 * nt + h)) & 1u ? __fadd_rn(__fmul_rn(p, factor), st.neg[nt][h])
                                               : fmaf(p, factor, st.neg[nt][h]);
        });
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[b][nt][e] = fast_exp2(y[b][nt][e]);
                st.l[nt][e & 1] += x[b][nt][e];
            }
}

// Weights x[4] of one head tile as B operands of the P V product, in PARTS parts of
// type E, each the last ones' remainder rounded: (b0, b1) = tokens 2 q4, 2 q4 + 1 and
// 8 + those, head r.  The remainders are exact.
template <typename E, int PARTS>
__device__ __forceinline__ void weight_parts(const float (&x)[4], uint32_t (&b)[PARTS][2])
{
    float rest[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
    for (int part = 0; part < PARTS; ++part)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t w = E::pack(rest[2 * k], rest[2 * k + 1]);
            b[part][k] = transpose8x8(w);
            const float2 f = E::unpack(w);
            rest[2 * k] -= f.x;
            rest[2 * k + 1] -= f.y;
        }
}

// ------------------------------------------------------------------ 16-bit block
// K and V slabs as TMA leaves them: boxes of 64 columns x 16 rows, 16-byte chunk
// c of row t at position c ^ (t % 8).  qb = the query rows as B operands.
// P goes in as parts of the pool's type: three of bf16 (2^-24; two, 2^-16, would show
// in the last bits of a result), two of fp16 (2^-22).
template <int D, bool BF16, int NT>
__device__ __forceinline__ void consume_16bit(uint32_t kb, const Queries<D, NT> &qs,
                                              State<D, NT> &st, uint32_t mask, float scale_log2,
                                              int lane)
{
    using E = Elem<BF16>;
    const auto &qb = qs.b;
    const int r = lane >> 2, q4 = lane & 3, mi = lane >> 3, r8 = lane & 7;
    const uint32_t vb = kb + 32 * D;
    float x[1][NT][4], c1[NT][4];        // two chains of products
    float (&c0)[NT][4] = x[0];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) c0[nt][e] = c1[nt][e] = 0.f;
    const int k_tok = ((mi & 1) << 3) + r8;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const int chunk = 2 * kk + (mi >> 1);
        uint32_t a[4];
        ldsm_x4(a, kb + (chunk >> 3) * kBoxBytes + k_tok * 128 + (((chunk & 7) ^ r8) << 4));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            E::mma(kk & 1 ? c1[nt] : c0[nt], a, qb[nt][kk][0], qb[nt][kk][1]);
    }
    float f[1][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        f[0][nt][0] = f[0][nt][1] = scale_log2;
#pragma unroll
        for (int e = 0; e < 4; ++e) c0[nt][e] += c1[nt][e];
    }
    const bool edge = mask != 0xffffu;   // the same for the warp: an edge of the visible part
    const uint32_t masks[1] = {mask};
    softmax_step<D, NT, 1>(st, x, f, masks, BF16 ? 0.f : kTop, lane);
    constexpr int kParts = BF16 ? 3 : 2;
    uint32_t w[NT][kParts][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) weight_parts<E, kParts>(c0[nt], w[nt]);
    // hidden tokens: their V rows may hold anything, and 0 * NaN is NaN
    const uint32_t two_lo = mask >> (2 * q4), two_hi = mask >> (2 * q4 + 8);
    const uint32_t keep_lo = (two_lo & 1u ? 0xffffu : 0u) | (two_lo & 2u ? 0xffff0000u : 0u);
    const uint32_t keep_hi = (two_hi & 1u ? 0xffffu : 0u) | (two_hi & 2u ? 0xffff0000u : 0u);
    const int v_tok = ((mi >> 1) << 3) + r8;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
        const int chunk = 2 * t + (mi & 1);
        uint32_t a[4];
        ldsm_x4_trans(a, vb + (chunk >> 3) * kBoxBytes + v_tok * 128 + (((chunk & 7) ^ r8) << 4));
        if (edge) {
            a[0] &= keep_lo;
            a[1] &= keep_lo;
            a[2] &= keep_hi;
            a[3] &= keep_hi;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int part = 0; part < kParts; ++part)
                E::mma(st.o[nt][t], a, w[nt][part][0], w[nt][part][1]);
    }
}

// ------------------------------------------------------------------- 8-bit block
// Byte u = code + 128 is the low mantissa of fp16 1024 + u (bits 0x6400 | u), so one
// byte permutation and one subtraction of 1152 make an fp16 pair of a byte pair.
// (Products that take the 1152 along, their sums starting from -1152 times the other
// operand's sum, need 64 instructions less per block and were 3 % faster where the SM
// is the limit; but they round at ten times the size of the terms, which showed in
// the last bits: 1.2 to 2 of 10,000 of a bf16 result's norm against the plain form's.
// The bytes as fp16 subnormals, u 2^-24, with an offset of 128: as exact as the
// subtraction but where one weight is far above the rest, and 1 to 3 % faster.)
__device__ __forceinline__ uint32_t centred(uint32_t w)
{
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(0x64806480u));   // (1152, 1152)
    return d;
}
__device__ __forceinline__ uint32_t codes_lo(uint32_t w)     // bytes 0 and 1
{
    return centred(__byte_perm(w, 0x64646464u, 0x4140));
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w)     // bytes 2 and 3
{
    return centred(__byte_perm(w, 0x64646464u, 0x4342));
}

// Offset of 16-byte chunk j of token t in the K or V codes (pagedkv.h).
template <int D>
__device__ __forceinline__ int chunk_at(int t, int j)
{
    return ((t * D) >> 7) * 128 + ((j ^ ((t & 1) << 2) ^ (((t >> 1) & 3) << 1)) << 4);
}

// Codes are exact in fp16, so both products run on fp16 operands; the block's
// two scales stay out of them: K's multiplies the scores, V's the block's
// product as it is added to the accumulator (weights then keep fp16's full
// precision whatever the scale), less the 2^kTop of the weights, which values
// near the largest bf16 leave no room for.  The reduction over dimensions
// may take them in any order, so lane (r, q4) takes whole 16-byte chunks q4
// (and q4 + 4) of tokens r and r + 8 as its A words, four dimensions to a step,
// and the queries were laid out alike; of V it takes dimensions D/8 r ..
// D/8 (r + 1) of its four tokens and pairs their bytes.
// P: two fp16 parts, which carry a weight to 2^-22 (one part, 2^-11, would show in a
// bf16 result: 8 of 10,000 of its norm against the plain form's; it was 2 % faster on
// grids that fill the GPU and 9 % where the SM is the limit).
// NB blocks at a time: their chains of dependent instructions overlap.
template <int D, int NT, int NB>
__device__ __forceinline__ void consume_b8(const uint8_t *const (&recs)[NB],
                                           const Queries<D, NT> &qs, State<D, NT> &st,
                                           const uint32_t (&masks)[NB], int lane)
{
    using H = Elem<false>;
    const auto &qb = qs.b;
    const auto &scale_row = qs.scale;
    const int r = lane >> 2, q4 = lane & 3;
    float x[NB][NT][4], f[NB][NT][2];
    float v_scale[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const uint8_t *rec = recs[b];
        const float2 scales = *reinterpret_cast<const float2 *>(rec + 32 * D);
        v_scale[b] = scales.y * kTopInverse;
        float c[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[nt][e] = 0.f;
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
            const uint4 wa = *reinterpret_cast<const uint4 *>(rec + chunk_at<D>(r, q4 + 4 * half));
            const uint4 wb = *reinterpret_cast<const uint4 *>(rec + chunk_at<D>(r + 8, q4 + 4 * half));
            const uint32_t ua[4] = {wa.x, wa.y, wa.z, wa.w}, ub[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a[4] = {codes_lo(ua[i]), codes_lo(ub[i]), codes_hi(ua[i]),
                                       codes_hi(ub[i])};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    H::mma(c[nt], a, qb[nt][4 * half + i][0], qb[nt][4 * half + i][1]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int h = 0; h < 2; ++h) f[b][nt][h] = scales.x * scale_row[nt][h];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[b][nt][e] = c[nt][e];
        }
    }
    softmax_step<D, NT, NB>(st, x, f, masks, kTop, lane);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        uint32_t p[NT][2][2];            // the weights' parts
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) weight_parts<H, 2>(x[b][nt], p[nt]);
        // words of tokens 2q4, 2q4 + 1, 2q4 + 8, 2q4 + 9: four dimensions each
        constexpr int kWords = D / 32;
        uint32_t w[4][kWords];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int t = 2 * q4 + (k & 1) + 8 * (k >> 1);
            const uint8_t *at = recs[b] + 16 * D;
            if constexpr (D == 128) {
                const uint4 v = *reinterpret_cast<const uint4 *>(at + chunk_at<D>(t, r));
                w[k][0] = v.x; w[k][1] = v.y; w[k][2] = v.z; w[k][3] = v.w;
            } else {
                const uint2 v =
                    *reinterpret_cast<const uint2 *>(at + chunk_at<D>(t, r >> 1) + 8 * (r & 1));
                w[k][0] = v.x; w[k][1] = v.y;
            }
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
#pragma unroll
            for (int pr = 0; pr < 2; ++pr) {          // dimensions 4i + 2 pr, 4i + 2 pr + 1
                const uint32_t sel = pr ? 0x7362 : 0x5140;
                const uint32_t p01 = __byte_perm(w[0][i], w[1][i], sel);
                const uint32_t p89 = __byte_perm(w[2][i], w[3][i], sel);
                const uint32_t a[4] = {codes_lo(p01), codes_hi(p01), codes_lo(p89), codes_hi(p89)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float c[4];
                    H::mma0(c, a, p[nt][0][0], p[nt][0][1]);
                    H::mma(c, a, p[nt][1][0], p[nt][1][1]);
                    float *o = st.o[nt][2 * i + pr];
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = fmaf(v_scale[b], c[e], o[e]);
                }
            }
        }
    }
}

// ------------------------------------------------------------------- query rows
// `rows`: the G rows of the kv head, global or shared memory.
template <int D, bool BF16, bool B8, int NT>
__device__ __forceinline__ void load_queries(Queries<D, NT> &qs, const typename Elem<BF16>::T *rows,
                                             int G, float scale_log2, int lane)
{
    using E = Elem<BF16>;
    const int r = lane >> 2, q4 = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int h = 8 * nt + r;
        qs.scale[nt][0] = qs.scale[nt][1] = scale_log2;
        if constexpr (!B8) {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(rows + h * D);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qs.b[nt][kk][0] = h < G ? w[8 * kk + q4] : 0u;
                qs.b[nt][kk][1] = h < G ? w[8 * kk + 4 + q4] : 0u;
            }
        } else {
#pragma unroll
            for (int half = 0; half < D / 64; ++half) {
                const uint4 *w = reinterpret_cast<const uint4 *>(rows + h * D + 16 * (q4 + 4 * half));
                const uint4 a = h < G ? w[0] : make_uint4(0u, 0u, 0u, 0u);
                const uint4 b = h < G ? w[1] : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) qs.b[nt][4 * half + (i >> 1)][i & 1] = u[i];
            }
            if constexpr (BF16) {
                // bf16 row -> fp16: times the power of two that puts its largest
                // magnitude into [2^14, 2^15); every value within 2^28 of it
                // converts exactly.  The inverse goes into the row's scale.
                float amax = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 f = E::unpack(qs.b[nt][kk][e]);
                        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
                const int ex = max(-112, ((__float_as_int(amax) >> 23) & 0xff) - 127 - 14);
                const float down = __int_as_float((127 - ex) << 23);
                const float up = __int_as_float((127 + ex) << 23);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 f = E::unpack(qs.b[nt][kk][e]);
                        qs.b[nt][kk][e] = Elem<false>::pack(f.x * down, f.y * down);
                    }
                qs.scale[nt][0] *= __shfl_sync(kFull, up, 8 * q4);
                qs.scale[nt][1] *= __shfl_sync(kFull, up, 8 * q4 + 4);
            }
        }
    }
}

// The sequence of place k when they are ordered by their visible blocks, longest
// first, in 32 classes (index order inside a class).  A grid of several waves
// then ends with its shortest pairs.  Every thread of the CTA calls it.
template <int THREADS>
__device__ __forceinline__ int longest_first(const Params &p, int k)
{
    __shared__ int count[32], found;
    __shared__ int warp_hits[THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto class_of = [&](int s) {
        const int L = p.context_lens[s];
        const int n = L < 0 || (int64_t)L > (int64_t)p.max_blocks_per_seq * kBlock
                          ? 0
                          : visible(L, p.window, p.sinks).n;
        return 31 - (int)((int64_t)n * 31 / p.most);
    };
    if (tid < 32) count[tid] = 0;
    if (tid == 0) found = 0;
    __syncthreads();
    for (int s = tid; s < p.num_seqs; s += THREADS) atomicAdd(&count[class_of(s)], 1);
    __syncthreads();
    // every warp for itself: the class that holds place k, and the place inside it
    const int c = count[lane];
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += y;
    }
    const int cls = __ffs(__ballot_sync(kFull, inc > k)) - 1;
    int left = k - __shfl_sync(kFull, inc - c, cls);
    for (int s0 = 0; s0 < p.num_seqs; s0 += THREADS) {
        const int s = s0 + tid;
        const bool hit = s < p.num_seqs && class_of(s) == cls;
        const unsigned hits = __ballot_sync(kFull, hit);
        __syncthreads();
        if (lane == 0) warp_hits[warp] = __popc(hits);
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += warp_hits[w];
            all += warp_hits[w];
        }
        if (hit && before + __popc(hits & ((1u << lane) - 1u)) == left) found = s;
        left -= all;
        if (left < 0) break;             // the same for the CTA
    }
    __syncthreads();
    return found;
}

// ------------------------------------------------------------ one cluster per pair
template <int D, bool BF16, bool B8, int NT, int W>
__global__ void __launch_bounds__(32 * W, Shape<D, B8, NT, W>::kMinBlocks)
    window_decode_kernel(const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const Params p)
{
    using SH = Shape<D, B8, NT, W>;
    constexpr int kWarps = W, kThreads = 32 * W;
    using E = Elem<BF16>;
    using T = typename E::T;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, q4 = lane & 3;
    uint8_t *ring = base + warp * SH::kWarpBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(base + SH::kBars) + warp * 8;
    float2 *ml = reinterpret_cast<float2 *>(base + SH::kMl);             // [warps + 1][16]
    __shared__ int abort_flags[kWarps];
    volatile int *abort_flag = &abort_flags[warp];
    if (lane == 0) {
        *abort_flag = 0;
        for (int i = 0; i < SH::kStages; ++i) mbar_init(smem_addr(&full[i]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    // a launch may overlap the end of the kernel before it: nothing of the call is
    // read above the wait (and by plain loads below it, which do not move above)
    griddep_launch_dependents();
    griddep_wait();

    const int C = p.ctas;
    const int64_t pair = blockIdx.x / C;
    const int rank = (int)(blockIdx.x - pair * C);
    int s = (int)(pair / p.num_kv_heads);
    const int g = (int)(pair - (int64_t)s * p.num_kv_heads);
    if (p.most > 0) s = longest_first<32 * W>(p, s);
    const int G = p.group;
    int L = p.context_lens[s];
    if (L < 0 || (int64_t)L > (int64_t)p.max_blocks_per_seq * kBlock) {
        if (threadIdx.x == 0) atomicOr(p.status, PKV_DEV_BAD_LEN);
        L = 0;
    }
    const Visible vis = visible(L, p.window, p.sinks);
    const int gw = rank * kWarps + warp, stride = C * kWarps;
    const int count = gw < vis.n ? (vis.n - 1 - gw) / stride + 1 : 0;   // this warp's blocks
    const int32_t *row = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
    auto load_ids = [&](int i0) {
        const int i = i0 + lane;
        return i < count ? row[vis.block(gw + i * stride)] : 0;
    };
    // bit l: the warp's block i0 + l holds hidden tokens
    auto edges_from = [&](int i0) {
        return __ballot_sync(kFull, vis.partial(vis.block(gw + (i0 + lane) * stride)));
    };
    int ids = load_ids(0), ids_next = load_ids(32);
    uint32_t bad = 0;
    auto issue = [&](int i) {            // the warp's i-th block into stage i % kStages
        if (i >= count) return;
        if ((i & 31) == 0 && i > 0) {
            ids = ids_next;
            ids_next = load_ids(i + 32);
        }
        const int id = __shfl_sync(kFull, ids, i & 31);
        const int slot = i % SH::kStages;
        const bool ok = id >= 0 && id < p.num_blocks;
        bad |= ok ? 0u : 1u;
        if (lane == 0) {
            const uint32_t fb = smem_addr(&full[slot]);
            const uint32_t dst = smem_addr(ring + slot * SH::kStageBytes);
            if (!ok) {
                atomicOr(p.status, PKV_DEV_BAD_BLOCK);
                mbar_arrive(fb);
            } else if constexpr (B8) {
                mbar_arrive_expect_tx(fb, SH::kCopyBytes);
                bulk_load(dst, p.kv + ((int64_t)id * p.num_kv_heads + g) * PKV_B8_RECORD_BYTES(D),
                          SH::kCopyBytes, fb);
            } else {
                mbar_arrive_expect_tx(fb, SH::kCopyBytes);
                const int y = (id * p.num_kv_heads + g) * kBlock;
#pragma unroll
                for (int bx = 0; bx < D / kBoxCols; ++bx) {
                    tma_load_2d(dst + bx * kBoxBytes, &tmK, bx * kBoxCols, y, fb);
                    tma_load_2d(dst + 32 * D + bx * kBoxBytes, &tmV, bx * kBoxCols, y, fb);
                }
            }
        }
    };
    for (int i = 0; i < SH::kStages; ++i) issue(i);

    Queries<D, NT> qs;
    load_queries<D, BF16, B8, NT>(qs, static_cast<const T *>(p.q) +
                                          ((int64_t)s * p.num_q_heads + (int64_t)g * G) * D,
                                  G, p.scale_log2, lane);
    State<D, NT> st;
    reset(st);
    // wait for the warp's i-th block; false (for the whole warp) when it gave up
    auto wait_block = [&](int i) {
        const bool landed = mbar_wait(smem_addr(&full[i % SH::kStages]),
                                      (uint32_t)(i / SH::kStages) & 1u, abort_flag, p.status);
        if (__all_sync(kFull, landed)) return true;
        // let the copies still in flight land first
        if (lane == 0) {
            for (int k = i; k < min(i + SH::kStages, count); ++k) {
                const unsigned long long t0 = globaltimer();
                while (!mbar_try_wait(smem_addr(&full[k % SH::kStages]),
                                      (uint32_t)(k / SH::kStages) & 1u))
                    if (globaltimer() - t0 > kTimeoutNs) break;
            }
        }
        __syncwarp();
        bad = 1u;
        return false;
    };
    auto stage_of = [&](int i) { return ring + (i % SH::kStages) * SH::kStageBytes; };
    uint32_t edges = 0;
    auto mask_of = [&](int i) {
        return (edges >> (i & 31)) & 1u ? vis.mask(vis.block(gw + i * stride)) : 0xffffu;
    };
    // the stages' next contents come through the async proxy: order this warp's
    // reads of them first
    auto released = [&]() {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
    };
    int i = 0;
    bool alive = true;
    if constexpr (B8 && NT == 1) {       // two blocks at a time (two head tiles: slower, 49.3 against
                                         // 48.3 us on 200 pairs of 16 fp16 heads)
        for (; i + 1 < count; i += 2) {
            if ((i & 31) == 0) edges = edges_from(i);
            alive = wait_block(i) && wait_block(i + 1);
            if (!alive) break;
            if (!bad) {
                const uint8_t *const recs[2] = {stage_of(i), stage_of(i + 1)};
                const uint32_t masks[2] = {mask_of(i), mask_of(i + 1)};
                consume_b8<D, NT, 2>(recs, qs, st, masks, lane);
            }
            released();
            issue(i + SH::kStages);
            issue(i + 1 + SH::kStages);
        }
    }
    for (; alive && i < count; ++i) {
        if ((i & 31) == 0) edges = edges_from(i);
        if (!wait_block(i)) break;
        if (!bad) {
            if constexpr (B8) {
                const uint8_t *const recs[1] = {stage_of(i)};
                const uint32_t masks[1] = {mask_of(i)};
                consume_b8<D, NT, 1>(recs, qs, st, masks, lane);
            } else {
                consume_16bit<D, BF16, NT>(smem_addr(stage_of(i)), qs, st, mask_of(i), p.scale_log2,
                                           lane);
            }
        }
        released();
        issue(i + SH::kStages);
    }

    // ---- the warp's piece, in its own ring: every copy into it has landed
    float *piece = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float l = st.l[nt][h];
            l += __shfl_xor_sync(kFull, l, 4);
            l += __shfl_xor_sync(kFull, l, 8);
            l += __shfl_xor_sync(kFull, l, 16);
            if constexpr (B8) l *= kTopInverse;          // as the accumulators
            const int head = 8 * nt + 2 * q4 + h;
            if (r == 0) ml[warp * kMaxHeads + head] = make_float2(st.m(nt, h), bad ? -1.f : l);
            float *dst = piece + head * SH::kRow;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) {
                if constexpr (B8) {
                    *reinterpret_cast<float2 *>(dst + D / 8 * r + 2 * t) =
                        make_float2(st.o[nt][t][h], st.o[nt][t][2 + h]);
                } else {
                    dst[16 * t + r] = st.o[nt][t][h];
                    dst[16 * t + r + 8] = st.o[nt][t][2 + h];
                }
            }
        }
    }
    __syncthreads();

    // ---- the CTA's warps: factors 2^(m_w - M), sums; a bad piece has sum -1
    T *out = static_cast<T *>(p.out) + ((int64_t)s * p.num_q_heads + (int64_t)g * G) * D;
    auto factor = [](float m, float M) { return m == -INFINITY ? 0.f : fast_exp2(m - M); };
    auto store = [&](int u, float4 a, float l, bool poisoned) {
        const float inv = 1.f / l;
        uint2 w = make_uint2(0u, 0u);     // no visible token, or a bad block: zeros
        if (vis.n > 0 && !poisoned) {
            w.x = E::pack(a.x * inv, a.y * inv);
            w.y = E::pack(a.z * inv, a.w * inv);
        }
        *reinterpret_cast<uint2 *>(out + 4 * u) = w;
    };
    const int units = G * (D / 4);        // four dimensions of a head each
    for (int u = threadIdx.x; u < units; u += kThreads) {
        const int h = u / (D / 4), d = 4 * (u - h * (D / 4));
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * kMaxHeads + h].x);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
        bool poisoned = false;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float2 v = ml[w * kMaxHeads + h];
            const float f = factor(v.x, M);
            const float4 x = *reinterpret_cast<const float4 *>(
                base + w * SH::kWarpBytes + (h * SH::kRow + d) * 4);
            a.x += x.x * f; a.y += x.y * f; a.z += x.z * f; a.w += x.w * f;
            l += v.y * f;
            poisoned |= v.y < 0.f;
        }
        if (C == 1) {
            store(u, a, l, poisoned);
        } else {                          // over warp 0's piece, which this thread alone reads here
            *reinterpret_cast<float4 *>(base + (h * SH::kRow + d) * 4) = a;
            if (d == 0) ml[kWarps * kMaxHeads + h] = make_float2(M, poisoned ? -1.f : l);
        }
    }
    if (C == 1) return;

    // ---- the cluster's CTAs: unit u goes to CTA u % C
    cluster_sync();
    for (int u = threadIdx.x * C + rank; u < units; u += kThreads * C) {
        const int h = u / (D / 4), d = 4 * (u - h * (D / 4));
        const uint32_t ml_at = smem_addr(ml + kWarps * kMaxHeads + h);
        const uint32_t o_at = smem_addr(base + (h * SH::kRow + d) * 4);
        float M = -INFINITY;
        for (int c = 0; c < C; ++c) M = fmaxf(M, cluster_load2(cluster_addr(ml_at, c)).x);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
        bool poisoned = false;
        for (int c = 0; c < C; ++c) {
            const float2 v = cluster_load2(cluster_addr(ml_at, c));
            const float4 x = cluster_load4(cluster_addr(o_at, c));
            const float f = factor(v.x, M);
            a.x += x.x * f; a.y += x.y * f; a.z += x.z * f; a.w += x.w * f;
            l += v.y * f;
            poisoned |= v.y < 0.f;
        }
        store(u, a, l, poisoned);
    }
    cluster_sync();                       // nobody leaves while its memory is read
}

// --------------------------------------------------------------------- host side
struct Variant {
    KernelFn fn;
    int smem, warps;
    int which;                 // index into the per-device cache
};

template <int D, bool B8, int W>
static Variant variant(bool bf16, bool wide)
{
    const int which = (D == 128) | B8 << 1 | bf16 << 2 | wide << 3 | (W > 4) << 4;
    if (wide)
        return bf16 ? Variant{&window_decode_kernel<D, true, B8, 2, W>, Shape<D, B8, 2, W>::kTotal, W, which}
                    : Variant{&window_decode_kernel<D, false, B8, 2, W>, Shape<D, B8, 2, W>::kTotal, W, which};
    return bf16 ? Variant{&window_decode_kernel<D, true, B8, 1, W>, Shape<D, B8, 1, W>::kTotal, W, which}
                : Variant{&window_decode_kernel<D, false, B8, 1, W>, Shape<D, B8, 1, W>::kTotal, W, which};
}

template <bool B8, int W>
static Variant variant(int D, bool bf16, bool wide)
{
    return D == 128 ? variant<128, B8, W>(bf16, wide) : variant<64, B8, W>(bf16, wide);
}

// What a variant can have on the current device, measured once per device.
constexpr int kMaxCluster = 16;
struct Limits {
    int sms, resident;                   // SMs; CTAs of the variant that fit at once
    int clusters[kMaxCluster + 1];       // clusters of c CTAs that fit at once (CTAs of 8 warps and more)
};

static bool limits(const Variant &v, Limits *out)
{
    constexpr int kMaxDev = 64, kVariants = 32;
    static std::mutex mu;
    static Limits cache[kMaxDev][kVariants];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return false;
    std::lock_guard<std::mutex> lock(mu);
    Limits &l = cache[dev][v.which];
    if (l.resident == 0) {
        int sms = 0, per_sm = 0;
        const void *fn = reinterpret_cast<const void *>(v.fn);
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem) !=
                cudaSuccess ||
            cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
                cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, 32 * v.warps, v.smem) !=
                cudaSuccess ||
            per_sm < 1)
            return false;
        for (int c = 1; c <= kMaxCluster && v.warps > 4; ++c) {
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = (unsigned)c;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)(c * sms));
            cfg.blockDim = dim3(32u * (unsigned)v.warps);
            cfg.dynamicSmemBytes = (size_t)v.smem;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) == cudaSuccess) l.clusters[c] = n;
            else (void)cudaGetLastError();           // a size that cannot be scheduled: 0
        }
        l.sms = sms;
        l.resident = sms * per_sm;
    }
    *out = l;
    return true;
}

// The most blocks a sequence can show (its length is known on the device only).
static int64_t most_blocks(int32_t maxb, int32_t window, int32_t sinks)
{
    return std::min<int64_t>(
        maxb, ((int64_t)window + 2 * kBlock - 2) / kBlock + ((int64_t)sinks + kBlock - 1) / kBlock);
}

static int launch(const pkv_pool *pool, bool want_b8, void *out, const void *q, const void *k_pool,
                  const void *v_pool, const int32_t *block_tables, int32_t maxb,
                  const int32_t *context_lens, int32_t num_seqs, int32_t num_q_heads, float scale,
                  int32_t window, int32_t sinks, int32_t *d_status, void *stream)
{
    PoolGeometry g;
    if (!pool_geometry(pool, &g)) return PKV_ERR_INVALID_ARG;
    if (want_b8 ? !is_b8(g) : !is_16bit(g)) return PKV_ERR_INVALID_ARG;
    if (num_seqs < 0 || num_q_heads <= 0 || maxb <= 0 || window < 1 || sinks < 0)
        return PKV_ERR_INVALID_ARG;
    if (num_q_heads % g.num_kv_heads) return PKV_ERR_INVALID_ARG;
    if (!(scale == scale) || scale == INFINITY || scale == -INFINITY) return PKV_ERR_INVALID_ARG;
    const int G = num_q_heads / g.num_kv_heads;
    if (g.block_size != kBlock || G > kMaxHeads || (g.head_dim != 64 && g.head_dim != 128))
        return PKV_ERR_UNSUPPORTED;
    if ((int64_t)maxb * kBlock > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    if (!want_b8 && (int64_t)g.num_blocks * g.num_kv_heads * g.block_size > (int64_t)1 << 31)
        return PKV_ERR_UNSUPPORTED;   // TMA row coordinate is a signed 32-bit value
    if (num_seqs == 0) return PKV_OK;
    if (!out || !q || !k_pool || (!want_b8 && !v_pool) || !block_tables || !context_lens || !d_status)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || (!want_b8 && !aligned16(v_pool)) ||
        ((uintptr_t)block_tables & 3u) || ((uintptr_t)context_lens & 3u) || ((uintptr_t)d_status & 3u))
        return PKV_ERR_INVALID_ARG;
    const bool bf = g.dtype == PKV_BF16 || g.dtype == PKV_B8_BF16, wide = G > 8;
    const int64_t pairs = (int64_t)num_seqs * g.num_kv_heads;
    const int64_t most = most_blocks(maxb, window, sinks);
    // Cluster size.  A cluster costs more to place the larger it is (a few
    // microseconds per wave of eights), so a pair is split only
    //  * while every CTA fits on the GPU at once and its warps have two blocks
    //    each: 32 pairs of 1,000 tokens 12.9 us split by 4 or 8, 19.1 unsplit;
    //    128 pairs 19.1 us unsplit to split by 3, 25 by 4 (past one wave), 31 by 8;
    //  * or, where a pair may show long runs of blocks, into about one and a half
    //    waves, for the GPU to stay busy to the end: 384 ragged pairs of up to
    //    6,000 tokens 68 us split by 2, 91 unsplit; 512 pairs of 4,000 tokens 126
    //    against 146; 1,280 pairs of up to 16,384 445 us unsplit, 455 split by 2.
    // (All with 9 us of event overhead, the L2 full of written data, 8-bit pools, 128
    // dimensions.)
    Variant v = want_b8 ? variant<true, 4>(g.head_dim, bf, wide) : variant<false, 4>(g.head_dim, bf, wide);
    Limits lim;
    if (!limits(v, &lim)) return PKV_ERR_CUDA;
    int C = 1;
    while (C < 8 && pairs * (C + 1) <= lim.resident && most >= 8 * (C + 1)) ++C;
    if (most >= 96 * C)
        while (C < 8 && 2 * pairs * C < 3 * lim.resident && most >= 48 * (C + 1)) ++C;
    if (pairs * 8 <= lim.sms && most >= 256) {
        // few long pairs: CTAs that take an SM each, in the largest clusters of
        // which every pair gets one at once (8 pairs of 60,000 tokens, as above:
        // 40 us with 12 CTAs of 12 warps, 50 with 8, 83 with 8 CTAs of four)
        v = want_b8 ? variant<true, 12>(g.head_dim, bf, wide) : variant<false, 8>(g.head_dim, bf, wide);
        if (!limits(v, &lim)) return PKV_ERR_CUDA;
        C = 1;
        for (int c = 2; c <= kMaxCluster; ++c)
            if (lim.clusters[c] >= pairs && most >= 2 * v.warps * c) C = c;
    }
    CUtensorMap tk = {}, tv = {};
    if (!want_b8 && (!decode::make_pool_map(&tk, k_pool, g) || !decode::make_pool_map(&tv, v_pool, g)))
        return PKV_ERR_CUDA;
    Params p;
    p.out = out;
    p.q = q;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.kv = static_cast<const uint8_t *>(k_pool);
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = g.num_kv_heads;
    p.group = G;
    p.max_blocks_per_seq = maxb;
    p.num_blocks = g.num_blocks;
    p.window = window;
    p.sinks = sinks;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.status = d_status;

    p.num_seqs = num_seqs;
    p.ctas = C;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // more than one wave, lengths not levelled by a window: longest pairs first
    // (every CTA looks at every length for it, so not for thousands of sequences,
    // whose many waves even out by themselves): the 1,280 pairs 445 us against 519 in
    // index order, the 384 68 against 89
    p.most = pairs * C > lim.resident && most == maxb && most >= 64 && num_seqs <= 512 ? (int)most : 0;
    if (pairs * C > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pairs * C));
    cfg.blockDim = dim3(32u * (unsigned)v.warps);
    cfg.dynamicSmemBytes = (size_t)v.smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, v.fn, tk, tv, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace window
}  // namespace pkv

extern "C" int paged_decode_attention_window(const pkv_pool *pool, void *out, const void *q,
                                             const void *k_pool, const void *v_pool,
                                             const int32_t *block_tables,
                                             int32_t max_blocks_per_seq,
                                             const int32_t *context_lens, int32_t num_seqs,
                                             int32_t num_q_heads, float scale, int32_t window,
                                             int32_t sinks, int32_t *d_status, void *stream)
{
    return pkv::window::launch(pool, false, out, q, k_pool, v_pool, block_tables,
                               max_blocks_per_seq, context_lens, num_seqs, num_q_heads, scale,
                               window, sinks, d_status, stream);
}

extern "C" int paged_decode_attention_b8(const pkv_pool *pool, void *out, const void *q,
                                         const void *kv_b8, const int32_t *block_tables,
                                         int32_t max_blocks_per_seq, const int32_t *context_lens,
                                         int32_t num_seqs, int32_t num_q_heads, float scale,
                                         int32_t window, int32_t sinks, int32_t *d_status,
                                         void *stream)
{
    if (window < 0) return PKV_ERR_INVALID_ARG;
    return pkv::window::launch(pool, true, out, q, kv_b8, nullptr, block_tables,
                               max_blocks_per_seq, context_lens, num_seqs, num_q_heads, scale,
                               window == 0 ? INT32_MAX : window, sinks, d_status, stream);
}
