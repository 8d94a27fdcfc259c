// Appending to the cache with the position rotation on the way, and the
// block-scaled 8-bit pools' write and read-back.
//
// Rotation of one head's row x at position p (cos, sin = the table's row p,
// half = rotary_dim / 2 entries each):
//   halves      (x[i], x[i + half]) -> (x[i] c - x[i + half] s, x[i + half] c + x[i] s)
//   neighbours  (x[2i], x[2i + 1])  -> (x[2i] c - x[2i + 1] s, x[2i + 1] c + x[2i] s)
// for i < half; dimensions from rotary_dim on stay as they are.  Each product
// and each sum is rounded to fp32 by itself (no fused multiply-add), so a
// result does not depend on how the compiler contracts the expression; the
// rotated value is rounded once more, to the row type (16-bit pools and
// queries) or to a code (8-bit pools, straight from fp32).
//
// Every value is read once and written once, so the kernels are bound by HBM
// (and, for a decode step's few rows, by the chain slot -> position -> table
// row -> store and the launch): 20,500 tokens of 32 query and 8 kv heads of 128 (505 MB)
// 78 to 81 us, 6.2 to 6.5 TB/s; into 8-bit blocks (463 MB) 75 us, 6.2 TB/s.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace append {

struct Params {
    const void *q, *k, *v;               // rows; token strides below, heads contiguous
    void *q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;   // elements
    const int32_t *positions;            // null: no rotation
    const float *cos_sin;                // [max_positions][rotary_dim]: cos, then sin
    const int64_t *slots;
    int32_t num_tokens, num_q_heads, num_kv_heads, max_positions, rotary_dim;
    int32_t block_size;
    int32_t block_shift, lane_shift;     // log2 of block_size and of head_dim / 16; -1: no power of two
    int64_t num_slots;
    uint4 *k_pool, *v_pool;              // 16-bit pools
    uint8_t *kv;                         // 8-bit records
    int32_t *status;
    int32_t write_blocks;                // 8-bit write: CTAs that write; the rest rotate queries
    int32_t parts;                       // of many tokens: CTAs that share a span's heads
    uint64_t minus_zeros;                // see mul2
};

// Every kernel here is launched with the programmatic attribute: it may be set up
// while the kernel before it in the stream ends, lets the next one do the same, and
// waits for the end of the one before it ahead of its first access to memory.
// What a call of this library may have written (rows, pools, scales) is read by plain
// or streaming loads (ld, ld.cs), not by __ldg: that one wants its data unchanged for
// the whole life of the kernel, and this life begins before the wait, while an append
// may still raise the scales that a read-back needs.  The cos/sin table is no call's
// output, and a kernel that does not let its successor start early (any other that
// fills the table) has ended before this life begins, so __ldg may read it (plain
// loads there: 13,300 tokens 17.8 us against 16.2, 20,500 into 8-bit blocks 103.5
// against 97.9).  A plain load does not move above the wait, the others when their
// pointer passed here.
__device__ __forceinline__ void begin()
{
    griddep_launch_dependents();
    griddep_wait();
}

template <typename T>
__device__ __forceinline__ void after_wait(T *&pointer)
{
    asm volatile("" : "+l"(pointer));
}

template <typename... P, typename... A>
static int launch(void (*fn)(P...), dim3 grid, int threads, int smem, cudaStream_t st, const A &...args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// A lane works on two 8-value chunks of a row.  Chunk pair i of the row: for
// the halves form the pairs' two sides (i and i + rotary_dim / 16) while i
// falls inside the rotated part, else two neighbouring chunks.
struct ChunkPair {
    int c0, c1;
    bool turned;
};

template <bool NEIGHBOURS>
__device__ __forceinline__ ChunkPair chunk_pair(int i, int rotary_dim)
{
    const int n = rotary_dim >> 4;       // chunk pairs of the rotated part
    if (i < n) return NEIGHBOURS ? ChunkPair{2 * i, 2 * i + 1, true} : ChunkPair{i, i + n, true};
    return ChunkPair{2 * i, 2 * i + 1, false};
}

constexpr uint64_t kMinusZeros = 0x8000000080000000ull;

// The kernels work on pairs of fp32 values in packed operations, half as many
// instructions.  A product and a sum are rounded each by itself; the compiler joins a
// packed product with the sum it feeds, so the product is written as a fused one whose
// addend, -0, it does not know: x y + (-0) is x y rounded once, signed zeros included.
__device__ __forceinline__ uint64_t mul2(const Params &p, uint64_t a, uint64_t b)
{
    return fma2f(a, b, p.minus_zeros);
}

// A lane's two chunks of a row.
struct Chunks {
    uint4 w0, w1;
};

// The 16 values of a chunk pair so that (a, b) are the pairs that a rotation turns.
// halves: a = the first chunk's values in order, b = the second's; neighbours: a = the
// even values of both chunks, b = the odd ones.  Entry m turns by angles 8i + 2m, + 1.
struct Values {
    uint64_t a[4], b[4];
};

template <bool BF16, bool NEIGHBOURS>
__device__ __forceinline__ Values unpack16(const uint4 &w0, const uint4 &w1)
{
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    Values v;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const float2 f = Elem<BF16>::unpack(w[NEIGHBOURS ? 2 * m : m]);
        const float2 g = Elem<BF16>::unpack(w[NEIGHBOURS ? 2 * m + 1 : 4 + m]);
        v.a[m] = NEIGHBOURS ? pack2f(f.x, g.x) : pack2f(f.x, f.y);
        v.b[m] = NEIGHBOURS ? pack2f(f.y, g.y) : pack2f(g.x, g.y);
    }
    return v;
}

// cs = the position's table row, in global memory or (SHARED) staged: there the cosines'
// float4s 0, 2, 4, ... come before 1, 3, 5, ..., the sines' likewise, so that
// neighbouring lanes read neighbouring float4s (other banks).
__device__ __forceinline__ int staged_at(int c, int half)     // place of a row's c-th float4
{
    const int quarter = half / 8, part = c >= 2 * quarter, e = c - 2 * quarter * part;
    return 2 * quarter * part + (e & 1) * quarter + (e >> 1);
}

struct Angles {
    uint64_t c[4], s[4];
};

template <bool SHARED>
__device__ __forceinline__ Angles angles(int i, int half, const float *cs)
{
    const ulonglong2 *c2 = reinterpret_cast<const ulonglong2 *>(cs) + (SHARED ? i : 2 * i);
    const ulonglong2 *s2 = c2 + half / 4;
    const int next = SHARED ? half / 8 : 1;
    const ulonglong2 ca = SHARED ? c2[0] : __ldg(c2), cb = SHARED ? c2[next] : __ldg(c2 + 1);
    const ulonglong2 sa = SHARED ? s2[0] : __ldg(s2), sb = SHARED ? s2[next] : __ldg(s2 + 1);
    return {{ca.x, ca.y, cb.x, cb.y}, {sa.x, sa.y, sb.x, sb.y}};
}

__device__ __forceinline__ void turn16(const Params &p, Values &v, const Angles &w)
{
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const uint64_t x = v.a[m], y = v.b[m];
        v.a[m] = sub2f(mul2(p, x, w.c[m]), mul2(p, y, w.s[m]));
        v.b[m] = add2f(mul2(p, y, w.c[m]), mul2(p, x, w.s[m]));
    }
}

// The values of the two chunks in order.
template <bool NEIGHBOURS>
__device__ __forceinline__ void in_order(const Values &v, float (&x)[16])
{
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const float2 a = unpack2f(v.a[m]), b = unpack2f(v.b[m]);
        x[NEIGHBOURS ? 4 * m : 2 * m] = a.x;
        x[NEIGHBOURS ? 4 * m + 2 : 2 * m + 1] = a.y;
        x[NEIGHBOURS ? 4 * m + 1 : 8 + 2 * m] = b.x;
        x[NEIGHBOURS ? 4 * m + 3 : 8 + 2 * m + 1] = b.y;
    }
}

// The 16-bit words of the two chunks.
template <bool BF16, bool NEIGHBOURS>
__device__ __forceinline__ Chunks pack16(const Values &v)
{
    using E = Elem<BF16>;
    uint32_t w[8];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const float2 a = unpack2f(v.a[m]), b = unpack2f(v.b[m]);
        w[NEIGHBOURS ? 2 * m : m] = NEIGHBOURS ? E::pack(a.x, b.x) : E::pack(a.x, a.y);
        w[NEIGHBOURS ? 2 * m + 1 : 4 + m] = NEIGHBOURS ? E::pack(a.y, b.y) : E::pack(b.x, b.y);
    }
    return {make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
}

// 16-bit pools (and, with heads_kv = 0, the queries of an 8-bit append): one thread per
// (token, R heads, chunk pair), heads in the order q, k, v: the R rows are under way
// together and share slot, position and the table's entries.  A thread reads what it
// writes and nothing else of q, so q_out may be q itself.
// R by measurement (R = 1, 2, 4): 20,500 tokens of 32/8 heads of 128, halves, 83, 79,
// 82 us, 4,000 18.7, 16.0, 15.8, 40,000 of 8/8 heads of 64 45.5, 42.0, 39.8; too few
// threads to fill the GPU at 4, 800 of 32/8 heads 4.3, 3.8, 4.9.  Neighbours (a thread's
// two chunks adjoin, so each of its accesses takes half a sector): 13,300 of 8/8 heads of
// 64 11.8, 12.9, 13.8, 20,000 of 32/8 41.8, 41.2, 42.4.
constexpr int kRowHeads = 4;
constexpr int64_t kRowHeadsFrom = 152 * 1024;             // threads with kRowHeads

template <bool BF16, bool NEIGHBOURS, int R>
__device__ __forceinline__ void append_rows(const Params &p, int D, int heads_kv, int cta, int ctas)
{
    const int lanes = D >> 4;                             // chunk pairs of a row
    const int turned_heads = p.num_q_heads + heads_kv, heads = turned_heads + heads_kv;
    const int groups = (heads + R - 1) / R, per_token = groups * lanes;
    // units first, first + step, ...: the token and the rest advance by fixed amounts
    const uint32_t first = (uint32_t)cta * blockDim.x + threadIdx.x;
    const uint32_t step = (uint32_t)ctas * blockDim.x;
    const int step_t = (int)(step / (uint32_t)per_token);
    const int step_w = (int)(step - (uint32_t)step_t * per_token);
    int64_t t = first / (uint32_t)per_token;
    int within = (int)(first - (uint32_t)t * per_token);
    for (; t < p.num_tokens; t += step_t, within += step_w) {
        if (within >= per_token) {
            within -= per_token;
            if (++t >= p.num_tokens) break;
        }
        const int group = p.lane_shift >= 0 ? within >> p.lane_shift : within / lanes;
        const int i = within - group * lanes;
        const ChunkPair cp = chunk_pair<NEIGHBOURS>(i, p.rotary_dim);
        const int64_t slot = p.slots[t];
        const int pos = p.positions[t];
        Chunks w[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int h = group + j * groups;             // neighbouring threads, neighbouring heads
            if (R > 1 && h >= heads) break;
            const uint16_t *row =
                h < p.num_q_heads ? static_cast<const uint16_t *>(p.q) + t * p.q_stride + h * D
                : h < turned_heads
                    ? static_cast<const uint16_t *>(p.k) + t * p.k_stride + (h - p.num_q_heads) * D
                    : static_cast<const uint16_t *>(p.v) + t * p.v_stride + (h - turned_heads) * D;
            w[j] = {reinterpret_cast<const uint4 *>(row)[cp.c0], reinterpret_cast<const uint4 *>(row)[cp.c1]};
        }
        if (slot < 0) continue;                           // no token here
        if (slot >= p.num_slots || pos < 0 || pos >= p.max_positions) {
            if (within == 0) atomicOr(p.status, slot >= p.num_slots ? PKV_DEV_BAD_SLOT : PKV_DEV_BAD_POS);
            continue;
        }
        if (cp.turned && group < turned_heads) {
            const Angles a =
                angles<false>(i, p.rotary_dim >> 1, p.cos_sin + (int64_t)pos * p.rotary_dim);
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (R > 1 && group + j * groups >= turned_heads) break;
                Values x = unpack16<BF16, NEIGHBOURS>(w[j].w0, w[j].w1);
                turn16(p, x, a);
                w[j] = pack16<BF16, NEIGHBOURS>(x);
            }
        }
        const int64_t block = p.block_shift >= 0 ? slot >> p.block_shift : slot / p.block_size;
        const int off = (int)(slot - block * p.block_size);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int h = group + j * groups, kh = h - p.num_q_heads, vh = h - turned_heads;
            if (R > 1 && h >= heads) break;
            uint4 *dst;
            if (kh < 0)
                dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.q_out) + t * p.q_out_stride + h * D);
            else
                dst = (vh < 0 ? p.k_pool : p.v_pool) +
                      ((block * heads_kv + (vh < 0 ? kh : vh)) * p.block_size + off) * (D >> 3);
            dst[cp.c0] = w[j].w0;
            dst[cp.c1] = w[j].w1;
        }
    }
}

template <bool BF16, bool NEIGHBOURS, int R>
__global__ void __launch_bounds__(256) append_rope_kernel(Params p, int D, int heads_kv)
{
    begin();
    after_wait(p.cos_sin);
    append_rows<BF16, NEIGHBOURS, R>(p, D, heads_kv, blockIdx.x, gridDim.x);
}

// ------------------------------------------------------- block-scaled 8-bit pools
// Byte of 16-byte chunk j of token t inside a record's K (or V) codes (see the
// layout in pagedkv.h): lines of 128 bytes, chunk positions rotated so that the
// attention kernel's wide shared-memory reads of either operand touch all banks.
__device__ __forceinline__ int b8_line(int t, int D) { return ((t * D) >> 7) * 128; }
__device__ __forceinline__ int b8_swizzle(int t) { return ((t & 1) << 6) ^ (((t >> 1) & 3) << 5); }
__device__ __forceinline__ int b8_chunk(int t, int j, int D) { return b8_line(t, D) + ((j * 16) ^ b8_swizzle(t)); }

// A table row staged in shared memory: this many floats apart beyond its own.
constexpr int kTablePad = 4;

// Values whose block maximum is below this store as zeros (scale 0): their
// reciprocal scale would leave the fp32 range.
constexpr float kB8Tiny = 0x1p-100f;

// Rounding to an integer, ties to even, of |x| <= 2^22: adding 1.5 * 2^23 puts
// the sum where the fp32 spacing is 1; its low byte is the integer's.
__device__ __forceinline__ uint32_t round_bits(float x)
{
    return __float_as_uint(__fadd_rn(x, 12582912.0f));
}

__device__ __forceinline__ uint32_t low_bytes(uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3)
{
    return __byte_perm(__byte_perm(b0, b1, 0x0040), __byte_perm(b2, b3, 0x0040), 0x5410);
}

// Codes of 16 values times inv as stored bytes (code + 128, where the sum that rounds
// puts the 128).  All values are at most 127 (1 + 2^-22) in size and round inside the
// range; in a block that holds an infinity or a NaN (odd) codes are clamped to
// [-127, 127] and NaN gives 0.
template <bool NEIGHBOURS>
__device__ __forceinline__ uint4 b8_codes16(const Params &p, const Values &v, float inv, bool odd)
{
    constexpr float kRound = 12582912.0f + 128.0f;
    uint32_t b[16];
    if (!odd) {
        const uint64_t inv2 = pack2f(inv, inv), round2 = pack2f(kRound, kRound);
        Values y;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            y.a[m] = add2f(mul2(p, v.a[m], inv2), round2);
            y.b[m] = add2f(mul2(p, v.b[m], inv2), round2);
        }
        float x[16];
        in_order<NEIGHBOURS>(y, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) b[e] = __float_as_uint(x[e]);
    } else {
        float x[16];
        in_order<NEIGHBOURS>(v, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            float y = __fmul_rn(x[e], inv);
            y = y == y ? fminf(fmaxf(y, -127.f), 127.f) : 0.f;
            b[e] = __float_as_uint(__fadd_rn(y, kRound));
        }
    }
    return make_uint4(low_bytes(b[0], b[1], b[2], b[3]), low_bytes(b[4], b[5], b[6], b[7]),
                      low_bytes(b[8], b[9], b[10], b[11]), low_bytes(b[12], b[13], b[14], b[15]));
}

// The largest of a and the values' sizes; NaN if any is.
__device__ __forceinline__ float max_abs_nan(float a, const Values &v)
{
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const float2 x = unpack2f(v.a[m]), y = unpack2f(v.b[m]);
        asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(a), "f"(x.x), "f"(x.y));
        asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(a), "f"(y.x), "f"(y.y));
    }
    return a;
}

// The same of two chunks of 16-bit values, which need no unpacking for it.  a = two
// such maxima; their signs mean nothing.
template <bool BF16>
__device__ __forceinline__ uint32_t max_abs_nan16(uint32_t a, uint32_t b)
{
    uint32_t m;
    if constexpr (BF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    else asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}

template <bool BF16>
__device__ __forceinline__ uint32_t max_abs_nan16(uint32_t a, const uint4 &w0, const uint4 &w1)
{
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int m = 0; m < 8; ++m) a = max_abs_nan16<BF16>(a, w[m]);
    return a;
}

__device__ __forceinline__ void copy16(uint4 *dst, const uint4 *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}

// Four stored bytes rounded to a larger scale (ratio = old / new <= 1).
__device__ __forceinline__ uint32_t b8_rescale4(uint32_t w, float ratio)
{
    uint32_t b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float c = (float)((int)((w >> (8 * k)) & 0xffu) - 128);
        b[k] = round_bits(__fmul_rn(c, ratio));
    }
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410) ^
           0x80808080u;
}

// One run of tokens t0 .. t0 + n - 1, whose slots are off0, off0 + 1, ... of one block,
// for one kv head, as a warp writes it: a row is D / 16 lanes of 16 values, a pass
// kRows rows.
template <int D>
struct Run {
    static constexpr int kLanes = D / 16, kRows = 32 / kLanes, kPasses = 16 / kRows;
    int t0, n, off0, h;
    int r, i;                            // the lane's row of a pass and its place in it
    uint8_t *rec;
    __device__ __forceinline__ Run(const Params &p, int t0_, int n_, int64_t slot, int h_, int lane)
        : t0(t0_), n(n_), off0((int)slot & (kBlock - 1)), h(h_), r(lane / kLanes), i(lane % kLanes),
          rec(p.kv + ((slot / kBlock) * p.num_kv_heads + h_) * PKV_B8_RECORD_BYTES(D))
    {
    }
    // call f(pass, the row's two chunks) for the lane's rows
    template <typename F>
    __device__ __forceinline__ void rows(const void *base, int64_t stride, const ChunkPair &cp, F &&f) const
    {
        const uint16_t *at = static_cast<const uint16_t *>(base) + (t0 + r) * stride + h * D;
#pragma unroll
        for (int k = 0; k < kPasses; ++k, at += kRows * stride)
            if (k * kRows + r < n)
                f(k, reinterpret_cast<const uint4 *>(at) + cp.c0, reinterpret_cast<const uint4 *>(at) + cp.c1);
    }
};

// Write K (part 0) or V (part 1) of a run.
//   scale = max(scale before, amax * rn(1 / 127)),  code = rn(x * rn(1 / scale))
// where "scale before" counts only when the run does not start the block (off0
// > 0).  When the scale grows, the codes of tokens 0 .. off0 - 1 are rounded to
// it: rn(code * rn(old / new)).
// raw(k) gives the two chunks of the lane's row of pass k, turn(k, values) rotates them
// (ROTATE), `keep` has the bits of the passes whose row is written.  A row stays packed
// between the maximum and the codes and is rotated for both.
template <bool BF16, bool NEIGHBOURS, bool ROTATE, int D, typename Raw, typename Turn>
__device__ __forceinline__ void b8_write_part(const Params &p, const Run<D> &u, int part,
                                              const ChunkPair &cp, uint32_t keep, int lane, Raw &&raw,
                                              Turn &&turn)
{
    constexpr int kPasses = Run<D>::kPasses;
    uint8_t *codes = u.rec + 16 * D * part;
    float *scale_at = reinterpret_cast<float *>(u.rec + 32 * D) + part;
    const float old = u.off0 > 0 ? *scale_at : 0.f;
    auto values = [&](int k) {
        const Chunks c = raw(k);
        Values v = unpack16<BF16, NEIGHBOURS>(c.w0, c.w1);
        if (ROTATE) turn(k, v);
        return v;
    };
    float amax = 0.f;
    uint32_t amax16 = 0u;
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        if (!((keep >> k) & 1u)) continue;
        if constexpr (ROTATE) {
            amax = max_abs_nan(amax, values(k));
        } else {
            const Chunks c = raw(k);
            amax16 = max_abs_nan16<BF16>(amax16, c.w0, c.w1);
        }
    }
    if constexpr (!ROTATE) {
        const float2 f = Elem<BF16>::unpack(amax16);
        asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(amax) : "f"(0.f), "f"(f.x), "f"(f.y));
    }
    // sizes are ordered as their bits are, infinity and NaN last
    constexpr float kMax = 0x1.fep127f;                       // the largest bf16
    amax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(amax)));
    const bool odd = !(amax <= kMax);                         // an infinity or a NaN
    if (odd) {                           // once more: NaN ignored, an infinity as kMax
        amax = 0.f;
#pragma unroll
        for (int k = 0; k < kPasses; ++k) {
            if (!((keep >> k) & 1u)) continue;
            float x[16];
            in_order<NEIGHBOURS>(values(k), x);
#pragma unroll
            for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
        }
        amax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(fminf(amax, kMax))));
    }
    if (amax < kB8Tiny) amax = 0.f;
    constexpr float kRcp127 = 0x1.020408p-7f;                 // rn(1 / 127)
    const float now = fmaxf(old, __fmul_rn(amax, kRcp127));
    if (u.off0 > 0 && now > old) {
        const float ratio = __fdiv_rn(old, now);
        for (int c = lane; c < u.off0 * Run<D>::kLanes; c += 32) {
            uint4 *at = reinterpret_cast<uint4 *>(
                codes + b8_chunk(c / Run<D>::kLanes, c % Run<D>::kLanes, D));
            uint4 v = *at;
            v.x = b8_rescale4(v.x, ratio);
            v.y = b8_rescale4(v.y, ratio);
            v.z = b8_rescale4(v.z, ratio);
            v.w = b8_rescale4(v.w, ratio);
            *at = v;
        }
    }
    if (lane == 0 && (u.off0 == 0 || now != old)) *scale_at = now;
    const float inv = now > 0.f ? __fdiv_rn(1.f, now) : 0.f;
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        if (!((keep >> k) & 1u)) continue;
        const int t = u.off0 + k * Run<D>::kRows + u.r, swizzle = b8_swizzle(t);
        uint8_t *line = codes + b8_line(t, D);
        const uint4 b = b8_codes16<NEIGHBOURS>(p, values(k), inv, odd);
        if (NEIGHBOURS || !ROTATE) {     // the two chunks are one of codes
            *reinterpret_cast<uint4 *>(line + ((cp.c0 * 8) ^ swizzle)) = b;
        } else {
            *reinterpret_cast<uint2 *>(line + (((cp.c0 >> 1) * 16) ^ swizzle) + 8 * (cp.c0 & 1)) =
                make_uint2(b.x, b.y);
            *reinterpret_cast<uint2 *>(line + (((cp.c1 >> 1) * 16) ^ swizzle) + 8 * (cp.c1 & 1)) =
                make_uint2(b.z, b.w);
        }
    }
}

// Write K and V of a run, or one of them (PARTS: bit 0 K, bit 1 V).  The rows wait in
// `stage`, those of V beside K in registers, all loaded before any is worked on.  SHARED:
// positions and cos_sin hold the rows of tokens t0, t0 + 1, ... in shared memory; else
// these are the call's arrays.  `ready` is called between the loads and the rest.
template <bool BF16, bool NEIGHBOURS, int D, bool SHARED, int PARTS, typename Ready>
__device__ __forceinline__ void b8_write_run(const Params &p, const Run<D> &u, int lane,
                                             const int *positions, const float *cos_sin, uint4 *stage,
                                             Ready &&ready)
{
    constexpr int kPasses = Run<D>::kPasses, kRows = Run<D>::kRows;
    const bool rotate = p.positions != nullptr;
    const ChunkPair plain = {2 * u.i, 2 * u.i + 1, false};
    const ChunkPair cp = rotate ? chunk_pair<NEIGHBOURS>(u.i, p.rotary_dim) : plain;
    auto to_stage = [&](int k, const uint4 *a, const uint4 *b) {
        copy16(stage + 64 * k + lane, a);                 // a lane stages what it will read itself
        copy16(stage + 64 * k + 32 + lane, b);
    };
    auto staged = [&](int k) { return Chunks{stage[64 * k + lane], stage[64 * k + 32 + lane]}; };
    if constexpr (PARTS & 1) u.rows(p.k, p.k_stride, cp, to_stage);
    Chunks v[kPasses];
    if constexpr (PARTS == 2) u.rows(p.v, p.v_stride, plain, to_stage);
    if constexpr (PARTS == 3)
        u.rows(p.v, p.v_stride, plain, [&](int k, const uint4 *a, const uint4 *b) { v[k] = {*a, *b}; });
    ready();
    uint32_t keep = 0u;                                   // rows to write
    int pos[kPasses];
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        const int j = k * kRows + u.r;
        pos[k] = j < u.n && rotate ? positions[(SHARED ? 0 : u.t0) + j] : 0;
        if (j < u.n) {
            if (pos[k] >= 0 && pos[k] < max(p.max_positions, 1)) keep |= 1u << k;
            else if (u.i == 0) atomicOr(p.status, PKV_DEV_BAD_POS);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if constexpr (PARTS & 1) {
        if (rotate)
            b8_write_part<BF16, NEIGHBOURS, true>(p, u, 0, cp, keep, lane, staged, [&](int k, Values &x) {
                const float *cs = cos_sin + (SHARED ? (int64_t)((k * kRows + u.r) * (D + kTablePad))
                                                    : (int64_t)pos[k] * p.rotary_dim);
                if (cp.turned) turn16(p, x, angles<SHARED>(u.i, p.rotary_dim >> 1, cs));
            });
        else
            b8_write_part<BF16, NEIGHBOURS, false>(p, u, 0, cp, keep, lane, staged, [](int, Values &) {});
    }
    if constexpr (PARTS & 2)
        b8_write_part<BF16, NEIGHBOURS, false>(
            p, u, 1, plain, keep, lane,
            [&](int k) {
                if constexpr (PARTS == 3) return v[k];
                else return staged(k);
            },
            [](int, Values &) {});
}

// The runs that begin among `span` tokens from tb on.  A run is a chain of tokens
// whose slots follow one another inside a block; lane l looks at token tb - 1 + l,
// so a run that begins at the span's last token is seen to its end.
struct Runs {
    int64_t slot;            // of token tb - 1 + lane
    unsigned links, leads;   // bit l: token tb - 1 + l goes on with a run, begins one
    __device__ __forceinline__ int length(int l) const     // of the run that token l begins
    {
        return __ffs(l < 31 ? ~(links >> (l + 1)) : ~0u);  // 1 + the links that follow
    }
};

__device__ __forceinline__ Runs find_runs(const Params &p, int64_t tb, int span, int lane, bool report)
{
    Runs r;
    const int64_t t = tb - 1 + lane;
    r.slot = t >= 0 && t < p.num_tokens ? p.slots[t] : -1;
    const int64_t prev = __shfl_up_sync(kFull, r.slot, 1);
    const bool valid = r.slot >= 0 && r.slot < p.num_slots;
    const unsigned mine = span == 16 ? 0x1fffeu : 0x2u;
    if ((__ballot_sync(kFull, r.slot >= p.num_slots) & mine) && lane == 0 && report)
        atomicOr(p.status, PKV_DEV_BAD_SLOT);
    const bool linked =
        lane > 0 && valid && prev >= 0 && prev + 1 == r.slot && r.slot % kBlock != 0;
    r.links = __ballot_sync(kFull, linked);
    r.leads = __ballot_sync(kFull, valid && !linked) & mine;
    return r;
}

// Few tokens: a warp takes one token, one kv head and K or V, and writes the run
// that begins there, if one does.
template <bool BF16, bool NEIGHBOURS, int D>
__global__ void __launch_bounds__(128, 6) append_b8_kernel(Params p)
{
    begin();
    after_wait(p.cos_sin);
    if ((int)blockIdx.x >= p.write_blocks) {              // queries only
        append_rows<BF16, NEIGHBOURS, 1>(p, D, 0, (int)blockIdx.x - p.write_blocks,
                                         (int)gridDim.x - p.write_blocks);
        return;
    }
    __shared__ uint4 stages[4 * 2 * D];
    const int lane = threadIdx.x & 31;
    uint4 *stage = stages + (threadIdx.x >> 5) * 2 * D;
    const int per_token = 2 * p.num_kv_heads;
    const int64_t units = (int64_t)p.num_tokens * per_token;
    for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); u < units;
         u += (int64_t)p.write_blocks * 4) {
        const int64_t t = u / per_token;
        const int rest = (int)(u - t * per_token);
        const Runs runs = find_runs(p, t, 1, lane, rest == 0);
        if (!runs.leads) continue;
        const int64_t s0 = __shfl_sync(kFull, runs.slot, 1);
        const Run<D> run(p, (int)t, runs.length(1), s0, rest >> 1, lane);
        if (rest & 1)
            b8_write_run<BF16, NEIGHBOURS, D, false, 2>(p, run, lane, p.positions, p.cos_sin, stage, [] {});
        else
            b8_write_run<BF16, NEIGHBOURS, D, false, 1>(p, run, lane, p.positions, p.cos_sin, stage, [] {});
    }
}

// Many tokens: a CTA takes a span of 16 and some of the kv heads (all, or a share of
// `parts`) and writes every run that begins there, the (run, kv head) units dealt to
// its warps.  The table rows of the tokens that they reach (up to 31) come to shared
// memory once for its heads, while the rows of the warps' first units are on their way.
constexpr int kSpanWarps = 8;
constexpr int kSpanTokens = 31;

template <bool BF16, bool NEIGHBOURS, int D>
__global__ void __launch_bounds__(32 * kSpanWarps, 3) append_b8_span_kernel(Params p)
{
    constexpr int kStride = D + kTablePad;                // floats of a staged table row
    extern __shared__ uint4 stages[];                     // [warps][16 rows x D / 8]
    __shared__ __align__(16) float table[kSpanTokens * kStride];
    __shared__ int positions[kSpanTokens + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint4 *stage = stages + warp * 2 * D;
    begin();
    after_wait(p.cos_sin);
    // write_blocks CTAs write, the others rotate queries, evenly mixed: an SM's writers
    // compute while its others wait for memory
    const int64_t before = (int64_t)blockIdx.x * p.write_blocks / gridDim.x;
    if ((int64_t)(blockIdx.x + 1) * p.write_blocks / gridDim.x == before) {
        append_rows<BF16, NEIGHBOURS, kRowHeads>(p, D, 0, (int)(blockIdx.x - before),
                                                 (int)gridDim.x - p.write_blocks);
        return;
    }
    const int spans = (int)(((int64_t)p.num_tokens + 15) / 16);
    for (int64_t w = before; w < (int64_t)spans * p.parts; w += p.write_blocks) {
        const int part = (int)(w % p.parts), tb = (int)(w / p.parts) * 16;
        const int head0 = p.num_kv_heads * part / p.parts;
        const int heads = p.num_kv_heads * (part + 1) / p.parts - head0;
        const Runs runs = find_runs(p, tb, 16, lane, part == 0 && warp == 0);
        const int n_leads = __popc(runs.leads), units = n_leads * heads;
        // of token tb - 1 + lane, asked for together with the slots
        const int at = tb - 1 + lane;
        const int lane_pos = p.positions && at >= 0 && at < p.num_tokens ? p.positions[at] : -1;
        auto fill = [&] {                                 // the table, up to the end of the last run
            if (!p.positions) return;
            const int last = 31 - __clz(runs.leads | 1u);
            const int n = runs.leads ? last - 1 + runs.length(last) : 0;
            const int per_row = p.rotary_dim / 4;
            for (int e0 = 32 * warp; e0 < n * per_row; e0 += 32 * kSpanWarps) {
                const int e = e0 + lane, t = e / per_row, c = e - t * per_row;
                const int pos = __shfl_sync(kFull, lane_pos, (t + 1) & 31);
                if (t < n && pos >= 0 && pos < p.max_positions)
                    *reinterpret_cast<float4 *>(table + t * kStride + 4 * staged_at(c, p.rotary_dim >> 1)) =
                        __ldg(reinterpret_cast<const float4 *>(p.cos_sin + (int64_t)pos * p.rotary_dim) + c);
            }
            if (warp == 0 && lane > 0) positions[lane - 1] = lane_pos;
            __syncthreads();
        };
        if (warp >= units) fill();
        for (int u = warp; u < units; u += kSpanWarps) {
            const int h = n_leads == 1 ? u : u / n_leads, k = u - h * n_leads;
            unsigned left = runs.leads;                   // the k-th run's first token
            for (int i = 0; i < k; ++i) left &= left - 1;
            const int l = __ffs(left) - 1;
            const int64_t s0 = __shfl_sync(kFull, runs.slot, l);
            const Run<D> run(p, tb - 1 + l, runs.length(l), s0, head0 + h, lane);
            b8_write_run<BF16, NEIGHBOURS, D, true, 3>(p, run, lane, positions + l - 1,
                                                       table + (l - 1) * kStride, stage, [&] {
                                                           if (u == warp) fill();
                                                       });
        }
        __syncthreads();                                  // the table may be filled anew
    }
}

// Records of blocks ids[0 .. n) as K and V rows [n][Hkv][16][D] of the row type: a unit
// is 8 codes of K and the same 8 of V, the e-th unit the e-th 16 bytes of either result;
// a thread has two units under way.  A code becomes fp32 as the low byte of 2^23 + byte.
// 203, 800 and 5,000 blocks of 8 heads of 128: 4.1, 10.3, 76 us (4.9, 7.7 from L2, 6.5
// TB/s); by 16 codes and integer conversions, one unit at a time, 6.2, 13.3, 78.
struct RecordUnit {
    int64_t e;
    uint2 k, v;
    float2 scales;
};

template <bool BF16>
__device__ __forceinline__ uint4 b8_values8(const uint2 &w, float scale)
{
    constexpr float kFirst = 8388608.0f;                  // 2^23
    const uint64_t zero2 = pack2f(-(kFirst + 128.f), -(kFirst + 128.f)), scale2 = pack2f(scale, scale);
    uint32_t out[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const uint32_t u = m < 2 ? w.x : w.y;
        const uint64_t x = pack2f(__uint_as_float(__byte_perm(u, __float_as_uint(kFirst), m & 1 ? 0x7652 : 0x7650)),
                                  __uint_as_float(__byte_perm(u, __float_as_uint(kFirst), m & 1 ? 0x7653 : 0x7651)));
        const float2 y = unpack2f(mul2f(add2f(x, zero2), scale2));
        out[m] = Elem<BF16>::pack(y.x, y.y);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

template <bool BF16, int D>
__global__ void __launch_bounds__(256)
    dequantize_kernel(const uint8_t *kv, const int32_t *ids, int32_t n, int32_t num_kv_heads,
                      int32_t num_blocks, uint4 *k_out, uint4 *v_out, int32_t *status)
{
    begin();
    after_wait(kv);
    constexpr int kUnits = 2 * D;                         // of a record
    const int64_t total = (int64_t)n * num_kv_heads * kUnits;
    auto load = [&](RecordUnit &u, int64_t e) {
        u.e = -1;
        if (e >= total) return;
        const int64_t record = e / kUnits;
        const int within = (int)(e % kUnits), t = within / (D / 8), half = within % (D / 8);
        const int64_t b = record <= UINT32_MAX ? (int64_t)((uint32_t)record / (uint32_t)num_kv_heads)
                                               : record / num_kv_heads;
        const int h = (int)(record - b * num_kv_heads);
        const int32_t id = ids[b];
        if (id < 0 || id >= num_blocks) {
            if (within == 0 && h == 0) atomicOr(status, PKV_DEV_BAD_BLOCK);
            return;
        }
        u.e = e;
        const uint8_t *rec = kv + ((int64_t)id * num_kv_heads + h) * PKV_B8_RECORD_BYTES(D);
        const uint8_t *codes = rec + b8_chunk(t, half >> 1, D) + 8 * (half & 1);
        u.k = __ldcs(reinterpret_cast<const uint2 *>(codes));
        u.v = __ldcs(reinterpret_cast<const uint2 *>(codes + 16 * D));
        u.scales = *reinterpret_cast<const float2 *>(rec + 32 * D);
    };
    auto finish = [&](const RecordUnit &u) {
        if (u.e < 0) return;
        k_out[u.e] = b8_values8<BF16>(u.k, u.scales.x);
        v_out[u.e] = b8_values8<BF16>(u.v, u.scales.y);
    };
    for (int64_t e = (int64_t)blockIdx.x * 512 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 512) {
        RecordUnit a, c;
        load(a, e);
        load(c, e + 256);
        finish(a);
        finish(c);
    }
}

// From this many values of K on, by spans of 16 tokens; below, a warp per token, head and
// part.  Prompts, by tokens and by spans: 32/8 heads of 128 1,500 tokens 12.1 and 12.6 us,
// 2,000 15.2 and 15.2, 3,000 20.9 and 16.9; 40/40 heads 320 tokens 11.2 and 11.4, 1,000
// 23.2 and 15.0; 8/2 heads of 64 6,000 tokens 9.8 and 11.2, 20,500 21.5 and 20.2.
constexpr int64_t kSpanValues = 1 << 21;
// A span's heads are shared by as many CTAs as fit at once (3 an SM): tokens of as many
// sequences as there are tokens make 16 runs a span, and one CTA for all heads takes long
// over them: 2,000 such tokens of 32/8 heads 55 us, 27.9 so (by tokens 26.5), 3,000 57.8
// and 38.3 (39.5); of 40/40 heads 1,000 212 and 50 (50).
constexpr int64_t kSpanCtas = 152 * 3;

template <bool BF16, bool NEIGHBOURS>
static int launch_rows(const Params &p, int D, int heads_kv, cudaStream_t st)
{
    const int heads = p.num_q_heads + 2 * heads_kv;
    const int64_t rows = (int64_t)p.num_tokens * (D / 16), many = rows * ((heads + kRowHeads - 1) / kRowHeads);
    const bool by_four = !NEIGHBOURS && many >= kRowHeadsFrom;
    const int64_t grid = std::min<int64_t>(((by_four ? many : rows * heads) + 255) / 256, 152 * 64);
    return launch(by_four ? &append_rope_kernel<BF16, NEIGHBOURS, NEIGHBOURS ? 1 : kRowHeads>
                          : &append_rope_kernel<BF16, NEIGHBOURS, 1>,
                  dim3((unsigned)grid), 256, 0, st, p, D, heads_kv);
}

template <bool BF16, bool NEIGHBOURS>
static int launch_b8(const Params &p0, int D, bool queries, cudaStream_t st)
{
    Params p = p0;
    const int64_t spans = ((int64_t)p.num_tokens + 15) / 16;
    if ((int64_t)p.num_tokens * p.num_kv_heads * D >= kSpanValues) {
        p.parts = (int32_t)std::max<int64_t>(1, std::min<int64_t>(kSpanCtas / spans, p.num_kv_heads));
        p.write_blocks = (int32_t)std::min<int64_t>(spans * p.parts, 152 * 64);
        int64_t grid = p.write_blocks;
        if (queries) {
            // kRowHeads rows at a time, four times a thread: 3,300, 8,000 and 20,500 tokens
            // 12.9, 34.5, 75.6 us; once 15.6, 36.7, 80.4; two rows 15.3, 37.8, 85.9; one
            // row 18.0, 43.6, 101
            const int64_t units =
                (int64_t)p.num_tokens * ((p.num_q_heads + kRowHeads - 1) / kRowHeads) * (D / 16);
            grid += std::min<int64_t>((units + 1023) / 1024, 152 * 64);
        }
        const int smem = kSpanWarps * 32 * D;
        void (*fn)(Params) = D == 128 ? &append_b8_span_kernel<BF16, NEIGHBOURS, 128>
                                      : &append_b8_span_kernel<BF16, NEIGHBOURS, 64>;
        // with the static part a little over the 48 KB of a plain launch
        if (cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return PKV_ERR_CUDA;
        return launch(fn, dim3((unsigned)grid), 32 * kSpanWarps, smem, st, p);
    }
    const int64_t units = (int64_t)p.num_tokens * 2 * p.num_kv_heads;
    p.write_blocks = (int32_t)std::min<int64_t>((units + 3) / 4, 152 * 64);
    int64_t grid = p.write_blocks;
    if (queries) {
        const int64_t threads = (int64_t)p.num_tokens * p.num_q_heads * (D / 16);
        grid += std::min<int64_t>((threads + 255) / 256, 152 * 64);
    }
    return launch(D == 128 ? &append_b8_kernel<BF16, NEIGHBOURS, 128>
                           : &append_b8_kernel<BF16, NEIGHBOURS, 64>,
                  dim3((unsigned)grid), 128, 0, st, p);
}

static int32_t log2_or_none(int32_t x)
{
    for (int32_t k = 0; k < 31; ++k)
        if (x == 1 << k) return k;
    return -1;
}

static bool rows_ok(const void *p, int64_t stride, int64_t width)
{
    return p && aligned16(p) && stride >= width && stride % 8 == 0;
}

}  // namespace append
}  // namespace pkv

extern "C" int kv_cache_write_rope(const pkv_pool *pool, void *q_out, int64_t q_out_stride,
                                   const void *q, int64_t q_stride, int32_t num_q_heads,
                                   const void *k_new, int64_t k_stride, const void *v_new,
                                   int64_t v_stride, const int32_t *positions,
                                   const float *cos_sin, int32_t max_positions, int32_t rotary_dim,
                                   int32_t interleaved, const int64_t *slot_mapping,
                                   int32_t num_tokens, void *k_pool, void *v_pool,
                                   int32_t *d_status, void *stream)
{
    using namespace pkv::append;
    pkv::PoolGeometry g;
    if (!pkv::pool_geometry(pool, &g) || num_tokens < 0 || num_q_heads < 0)
        return PKV_ERR_INVALID_ARG;
    const bool b8 = pkv::is_b8(g);
    if (!b8 && !pkv::is_16bit(g)) return PKV_ERR_INVALID_ARG;
    if (rotary_dim < 16 || rotary_dim > g.head_dim || max_positions <= 0)
        return PKV_ERR_INVALID_ARG;
    if (rotary_dim % 16 || g.head_dim % 16) return PKV_ERR_UNSUPPORTED;
    if (b8 && !pkv::b8_supported(g)) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (!k_pool || (!b8 && !v_pool) || !d_status || !positions || !cos_sin || !slot_mapping)
        return PKV_ERR_INVALID_ARG;
    const int64_t kw = (int64_t)g.num_kv_heads * g.head_dim, qw = (int64_t)num_q_heads * g.head_dim;
    if (!rows_ok(k_new, k_stride, kw) || !rows_ok(v_new, v_stride, kw) ||
        (num_q_heads > 0 &&
         (!rows_ok(q, q_stride, qw) || !rows_ok(q_out, q_out_stride, qw))))
        return PKV_ERR_INVALID_ARG;
    if (!pkv::aligned16(k_pool) || (!b8 && !pkv::aligned16(v_pool)) || !pkv::aligned16(cos_sin) ||
        ((uintptr_t)slot_mapping & 7u) || ((uintptr_t)positions & 3u) ||
        ((uintptr_t)d_status & 3u))
        return PKV_ERR_INVALID_ARG;
    Params p = {};
    p.q = q;
    p.k = k_new;
    p.v = v_new;
    p.q_out = q_out;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out_stride = q_out_stride;
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.slots = slot_mapping;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = g.num_kv_heads;
    p.max_positions = max_positions;
    p.rotary_dim = rotary_dim;
    p.block_size = g.block_size;
    p.block_shift = log2_or_none(g.block_size);
    p.lane_shift = log2_or_none(g.head_dim / 16);
    p.num_slots = (int64_t)g.num_blocks * g.block_size;
    p.k_pool = static_cast<uint4 *>(k_pool);
    p.v_pool = static_cast<uint4 *>(v_pool);
    p.kv = static_cast<uint8_t *>(k_pool);
    p.status = d_status;
    p.minus_zeros = kMinusZeros;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool bf = g.dtype == PKV_BF16 || g.dtype == PKV_B8_BF16, nb = interleaved != 0;
    if (b8) {
        const bool q = num_q_heads > 0;
        return bf ? (nb ? launch_b8<true, true>(p, g.head_dim, q, st)
                        : launch_b8<true, false>(p, g.head_dim, q, st))
                  : (nb ? launch_b8<false, true>(p, g.head_dim, q, st)
                        : launch_b8<false, false>(p, g.head_dim, q, st));
    }
    return bf ? (nb ? launch_rows<true, true>(p, g.head_dim, g.num_kv_heads, st)
                    : launch_rows<true, false>(p, g.head_dim, g.num_kv_heads, st))
              : (nb ? launch_rows<false, true>(p, g.head_dim, g.num_kv_heads, st)
                    : launch_rows<false, false>(p, g.head_dim, g.num_kv_heads, st));
}

extern "C" int kv_cache_write_b8(const pkv_pool *pool, const void *k_new, const void *v_new,
                                 const int64_t *slot_mapping, int32_t num_tokens, void *kv_b8,
                                 int32_t *d_status, void *stream)
{
    using namespace pkv::append;
    pkv::PoolGeometry g;
    if (!pkv::pool_geometry(pool, &g) || num_tokens < 0 || !pkv::is_b8(g)) return PKV_ERR_INVALID_ARG;
    if (!pkv::b8_supported(g)) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (!k_new || !v_new || !slot_mapping || !kv_b8 || !d_status) return PKV_ERR_INVALID_ARG;
    if (!pkv::aligned16(k_new) || !pkv::aligned16(v_new) || !pkv::aligned16(kv_b8) ||
        ((uintptr_t)slot_mapping & 7u) || ((uintptr_t)d_status & 3u))
        return PKV_ERR_INVALID_ARG;
    Params p = {};
    p.k = k_new;
    p.v = v_new;
    p.k_stride = p.v_stride = (int64_t)g.num_kv_heads * g.head_dim;
    p.slots = slot_mapping;
    p.num_tokens = num_tokens;
    p.num_kv_heads = g.num_kv_heads;
    p.block_size = g.block_size;
    p.num_slots = (int64_t)g.num_blocks * g.block_size;
    p.kv = static_cast<uint8_t *>(kv_b8);
    p.status = d_status;
    p.minus_zeros = kMinusZeros;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return g.dtype == PKV_B8_BF16 ? launch_b8<true, false>(p, g.head_dim, false, st)
                                  : launch_b8<false, false>(p, g.head_dim, false, st);
}

extern "C" int kv_dequantize_blocks(const pkv_pool *pool, const int32_t *ids, int32_t n,
                                    const void *kv_b8, void *k_out, void *v_out, int32_t *d_status,
                                    void *stream)
{
    using namespace pkv::append;
    pkv::PoolGeometry g;
    if (!pkv::pool_geometry(pool, &g) || n < 0 || !pkv::is_b8(g)) return PKV_ERR_INVALID_ARG;
    if (!pkv::b8_supported(g)) return PKV_ERR_UNSUPPORTED;
    if (n == 0) return PKV_OK;
    if (!ids || !kv_b8 || !k_out || !v_out || !d_status) return PKV_ERR_INVALID_ARG;
    if (!pkv::aligned16(kv_b8) || !pkv::aligned16(k_out) || !pkv::aligned16(v_out) ||
        ((uintptr_t)ids & 3u) || ((uintptr_t)d_status & 3u))
        return PKV_ERR_INVALID_ARG;
    const int64_t total = (int64_t)n * g.num_kv_heads * g.head_dim * 2;      // units
    const int64_t grid = std::min<int64_t>((total + 511) / 512, 152 * 64);
    const bool bf = g.dtype == PKV_B8_BF16;
    auto fn = g.head_dim == 128 ? (bf ? &dequantize_kernel<true, 128> : &dequantize_kernel<false, 128>)
                                : (bf ? &dequantize_kernel<true, 64> : &dequantize_kernel<false, 64>);
    return launch(fn, dim3((unsigned)grid), 256, 0, static_cast<cudaStream_t>(stream),
                  static_cast<const uint8_t *>(kv_b8), ids, n, g.num_kv_heads, g.num_blocks,
                  static_cast<uint4 *>(k_out), static_cast<uint4 *>(v_out), d_status);
}
