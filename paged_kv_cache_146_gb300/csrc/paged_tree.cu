// Attention of trees of drafted tokens over the paged cache (sm_103a).
//
// Row r, drafted token i of its sequence (context L, n drafted tokens, base = L - n):
//   x_j = scale <q, K_j>,  out = sum_j softmax(x)_j V_j   over the j that it sees:
//   j < base,  or  base <= j < L and bit j - base of its mask is set.
//
// One warp per row and query head, a key at a time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace tree {

constexpr int kMaxWords = 32;

struct Params {
    void *out;
    const void *q, *k_pool, *v_pool;
    const int32_t *block_tables, *query_start, *context_lens;
    const uint32_t *mask;
    int32_t words, num_seqs, num_tokens, num_q_heads, num_kv_heads, max_blocks_per_seq, num_blocks;
    float scale_log2;
    int32_t *status;
};

template <int D, bool BF16>
__global__ void __launch_bounds__(256) tree_rows_kernel(const Params p)
{
    using E = Elem<BF16>;
    using T = typename E::T;
    constexpr int kPer = D / 32;
    const int s = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r0 = p.query_start[s], r1 = p.query_start[s + 1], L = p.context_lens[s], n = r1 - r0;
    if (!(0 <= r0 && r0 <= r1 && r1 <= p.num_tokens)) {
        if (threadIdx.x == 0) atomicOr(p.status, PKV_DEV_BAD_LEN);
        return;
    }
    const int32_t *row = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
    bool dead = L < n || (int64_t)L > (int64_t)p.max_blocks_per_seq * kBlock || n > 32 * p.words;
    if (dead && threadIdx.x == 0) atomicOr(p.status, PKV_DEV_BAD_LEN);
    if (!dead && n > 0) {
        bool bad = false;
        for (int b = threadIdx.x; b < (L + kBlock - 1) / kBlock; b += blockDim.x)
            bad |= row[b] < 0 || row[b] >= p.num_blocks;
        if (__syncthreads_or(bad)) {
            dead = true;
            if (threadIdx.x == 0) atomicOr(p.status, PKV_DEV_BAD_BLOCK);
        }
    }
    const int G = p.num_q_heads / p.num_kv_heads;
    for (int e = blockIdx.y * 8 + warp; e < n * p.num_q_heads; e += gridDim.y * 8) {
        const int i = e / p.num_q_heads, h = e - i * p.num_q_heads, g = h / G;
        const int64_t at = ((int64_t)(r0 + i) * p.num_q_heads + h) * D + lane * kPer;
        float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int d = 0; d < kPer; ++d) {
            q[d] = (float)static_cast<const T *>(p.q)[at + d];
            o[d] = 0.f;
        }
        for (int j = 0; j < (dead ? 0 : L); ++j) {
            const int d0 = j - (L - n);
            if (d0 >= 0 && !((p.mask[(int64_t)(r0 + i) * p.words + (d0 >> 5)] >> (d0 & 31)) & 1u)) continue;
            const int64_t kv =
                (((int64_t)row[j / kBlock] * p.num_kv_heads + g) * kBlock + j % kBlock) * D + lane * kPer;
            float x = 0.f;
#pragma unroll
            for (int d = 0; d < kPer; ++d) x = fmaf(q[d], (float)static_cast<const T *>(p.k_pool)[kv + d], x);
#pragma unroll
            for (int f = 16; f > 0; f >>= 1) x += __shfl_xor_sync(kFull, x, f);
            x *= p.scale_log2;
            const float now = x != x ? x : fmaxf(m, x), f = m == now ? 1.f : exp2f(m - now);
            const float w = x == -INFINITY ? 0.f : exp2f(x - now);
            l = l * f + w;
#pragma unroll
            for (int d = 0; d < kPer; ++d)
                o[d] = fmaf(w, (float)static_cast<const T *>(p.v_pool)[kv + d], o[d] * f);
            m = now;
        }
#pragma unroll
        for (int d = 0; d < kPer; ++d)
            static_cast<T *>(p.out)[at + d] = E::from_float(l == 0.f ? 0.f : o[d] / l);
    }
}

}  // namespace tree
}  // namespace pkv

extern "C" size_t paged_tree_workspace_bytes(int32_t num_tokens, int32_t num_q_heads,
                                             int32_t num_kv_heads, int32_t head_dim)
{
    if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
        num_q_heads / num_kv_heads > 16 || (head_dim != 64 && head_dim != 128))
        return 0;
    return 256;
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
    if (g.block_size != pkv::kBlock || num_q_heads / g.num_kv_heads > 16 ||
        (g.head_dim != 64 && g.head_dim != 128))
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !query_start || !context_lens ||
        !tree_mask || !workspace || !d_status)
        return PKV_ERR_INVALID_ARG;
    if (!pkv::aligned16(out) || !pkv::aligned16(q) || !pkv::aligned16(k_pool) ||
        !pkv::aligned16(v_pool) || ((uintptr_t)workspace & 255u) ||
        ((uintptr_t)block_tables & 3u) || ((uintptr_t)query_start & 3u) ||
        ((uintptr_t)context_lens & 3u) || ((uintptr_t)tree_mask & 3u) || ((uintptr_t)d_status & 3u))
        return PKV_ERR_INVALID_ARG;
    if (workspace_bytes <
        paged_tree_workspace_bytes(num_tokens, num_q_heads, g.num_kv_heads, g.head_dim))
        return PKV_ERR_INVALID_ARG;
    if ((int64_t)g.num_blocks * g.num_kv_heads * g.block_size > (int64_t)1 << 31)
        return PKV_ERR_UNSUPPORTED;
    Params prm;
    prm.out = out;
    prm.q = q;
    prm.k_pool = k_pool;
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
    prm.max_blocks_per_seq = max_blocks_per_seq;
    prm.num_blocks = g.num_blocks;
    prm.scale_log2 = scale * 1.4426950408889634f;
    prm.status = d_status;
    const bool bf16 = g.dtype == PKV_BF16;
    auto fn = g.head_dim == 128 ? (bf16 ? &tree_rows_kernel<128, true> : &tree_rows_kernel<128, false>)
                                : (bf16 ? &tree_rows_kernel<64, true> : &tree_rows_kernel<64, false>);
    fn<<<dim3((unsigned)num_seqs, 32), 256, 0, (cudaStream_t)stream>>>(prm);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
