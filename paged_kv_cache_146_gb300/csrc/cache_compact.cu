// The accepted path of a tree of drafted tokens, and moving kept tokens of the cache
// together.
#include <cuda_runtime.h>

#include <algorithm>

#include "pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace compact {

// Every kernel here is launched with the programmatic attribute: it may be set up while
// the kernel before it ends, and waits for that end ahead of its first access to memory.
template <typename... P, typename... A>
static int launch(void (*fn)(P...), dim3 grid, int threads, cudaStream_t st, const A &...args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// ------------------------------------------------------------------- accepted path
struct Trees {
    const void *tokens, *targets;
    const int32_t *parents, *query_start, *first;
    int32_t num_seqs, num_tokens;
    int32_t *kept, *num_kept;
    void *next_tokens;
    int32_t *status;
};

// A warp per sequence.  Trees of up to kHeld nodes are read at once, one latency for all, and
// walked in registers: a step takes the target from the lane that holds the last kept node and
// asks all nodes whether they are its child and hold that token.  256 trees of 21 to 64 nodes: 3.9
// us back to back (5.7 when each step read its nodes from L1; one small tree 2.6, the launch).
// Larger trees read theirs at each step: 64 of 129 to 400 nodes 7.0, 8 of 1,024 10.7.
constexpr int kAcceptWarps = 4, kSteps = 4, kHeld = 32 * kSteps;

template <typename T>
__global__ void __launch_bounds__(32 * kAcceptWarps) tree_accept_kernel(const Trees p)
{
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int s = blockIdx.x * kAcceptWarps + (threadIdx.x >> 5);
    if (s >= p.num_seqs) return;
    const int r0 = p.query_start[s], r1 = p.query_start[s + 1], first = p.first[s];
    const bool rows_ok = 0 <= r0 && r0 <= r1 && r1 <= p.num_tokens;
    const int n = rows_ok ? r1 - r0 : 0;
    const bool fits = rows_ok && first >= 0 && first <= INT32_MAX - n;
    const T *tokens = static_cast<const T *>(p.tokens) + (n ? r0 : 0);
    const T *targets = static_cast<const T *>(p.targets) + (n ? r0 : 0);
    const int32_t *parents = p.parents + (n ? r0 : 0);
    int32_t *kept = p.kept + (n ? r0 : 0);
    int num = 0;
    T next = (T)-1;
    bool bad = false;
    if (n <= kHeld) {
        int up[kSteps], path[kSteps];                    // node lane + 32 k; entry lane + 32 k
        T token[kSteps], target[kSteps];
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int i = lane + 32 * k;
            up[k] = i < n ? parents[i] : -1;
            token[k] = i < n ? tokens[i] : (T)0;
            target[k] = i < n ? targets[i] : (T)0;
            path[k] = 0;
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) bad |= up[k] < -1 || (up[k] >= lane + 32 * k && lane + 32 * k < n);
        bad = __any_sync(kFull, bad);                    // (node 0: -1)
        for (int at = 0; fits && !bad && at >= 0 && at < n;) {
            T mine = target[0];
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                mine = at >= 32 * k ? target[k] : mine;
                path[k] = num == lane + 32 * k ? at : path[k];
            }
            next = __shfl_sync(kFull, mine, at & 31);
            ++num;
            int child = -1;
#pragma unroll
            for (int k = kSteps - 1; k >= 0; --k) {
                const unsigned hits = __ballot_sync(kFull, lane + 32 * k < n && up[k] == at && token[k] == next);
                if (hits) child = 32 * k + __ffs(hits) - 1;
            }
            at = child;
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int i = lane + 32 * k;
            if (i < n) kept[i] = i < num ? first + path[k] : -1;
        }
    } else {
        for (int i = lane; i < n; i += 32) {
            const int above = parents[i];
            bad |= above < -1 || above >= i;
            kept[i] = -1;
        }
        bad = __any_sync(kFull, bad);
        __syncwarp();                                    // the -1 before the positions
        for (int at = 0; fits && !bad && at >= 0;) {
            if (lane == 0) kept[num] = first + at;
            ++num;
            next = targets[at];
            int child = -1;
            for (int i0 = (at + 1) & ~31; i0 < n && child < 0; i0 += 32) {
                const int i = i0 + lane;
                const unsigned hits = __ballot_sync(kFull, i < n && parents[i] == at && tokens[i] == next);
                if (hits) child = i0 + __ffs(hits) - 1;
            }
            at = child;
        }
    }
    if (lane == 0) {
        if (!fits || bad) atomicOr(p.status, fits ? PKV_DEV_BAD_TREE : PKV_DEV_BAD_LEN);
        p.num_kept[s] = num;
        static_cast<T *>(p.next_tokens)[s] = next;
    }
}

// ------------------------------------------------------------------- moving tokens
struct Moves {
    const int32_t *block_tables, *kept, *kept_start, *num_kept, *first;
    int32_t max_blocks_per_seq, num_entries, num_kv_heads, block_size, num_blocks;
    int32_t chunks;                      // 16-byte chunks of a row
    int32_t part_chunks, parts;          // of them a CTA's, and CTAs that share a row
    int32_t pairs;                       // (kv head, K or V) of a CTA
    int32_t batch;                       // tokens of a batch
    int32_t units;                       // shares of all sequences' rows, at most, see parts_of
    uint4 *k_pool, *v_pool;
    int32_t *status;
};

// A CTA takes a sequence, some of its (kv head, K or V) pairs, and a share of each row; nothing
// else reads or writes these bytes.  It goes through the kept tokens in order, a batch at a time:
// all of the batch's rows are read, then written.  A destination is never above its source and
// sources rise, so what a batch writes is no source of a later one.
// What bounds it is how many rows are under way at once and the instructions of a chunk: places are
// looked up once for a CTA and a batch ahead of the rows, the list is read two ahead.  Nine caches
// of up to 16,384 tokens that keep 40,000 in all (305 MB moved): 64 us, 4.8 TB/s (floor 45; the
// longest list's 8,000 tokens set the end); before the last steps it was 71 us, 93 with whole rows to
// a CTA, four times as long when each thread looked up its rows' places.
//
// Threads, chunks of a thread under way, tokens of a batch at most, CTAs to an SM.  The host
// chooses by the lists' room, num_entries / num_seqs, as what is kept of it is on the device: right
// for lists that fill their room, while the few kept nodes of wide trees go to Many (96 trees of 64
// nodes of which 1 to 6 are kept 7.9 us, 256 18.0; of 16 nodes, Brief, 3.5 and 7.2).
//   Many: what is under way on an SM is the same as in Few, but a CTA waits for its slowest row, so
//     many small ones end earlier (100 caches of 300 to 900 tokens 59 us, 77 with Few, then).
//   Uneven: up to 32 long lists share their rows by length (10 lists of 1,000 to 14,000 tokens 113
//     us, 140 with Many; below kLongList entries on average the search costs more than it gives, 20
//     lists of 130: 9.8 us against 6.6, then).
//   Few: calls with no more CTAs than SMs (a cache of 16,000 tokens: 64; 29 us, 56 with Many).
//   Brief: room of up to kBriefList entries, far less than a batch, several pairs to a CTA (96 lists of
//     up to 6 in 16: 3.6 us, 8.0 with Many; 64 lists of 20 to 100: 7.5, 6.2 with Many).
struct Many {
    static constexpr bool kByLength = false, kPairs = false;
    static constexpr int kThreads = 256, kDepth = 8, kBatch = 512, kCtas = 3;
};
struct Uneven : Many {
    static constexpr bool kByLength = true;
};
struct Few {
    static constexpr bool kByLength = false, kPairs = false;
    static constexpr int kThreads = 1024, kDepth = 4, kBatch = 960, kCtas = 1;   // 46 KB of places
};
struct Brief {
    static constexpr bool kByLength = false, kPairs = true;
    static constexpr int kThreads = 256, kDepth = 4, kBatch = 512, kCtas = 3;
};
constexpr int kFewCtas = 152, kBriefList = 32, kLongList = 512, kManyCtas = 152 * Many::kCtas;
constexpr int kMoveCtas = 608;           // rows are shared until there are four CTAs for an SM

struct Place {
    int64_t from, to;                    // chunks of the pool before kv head 0's row, -1: does not move
};

// CTAs that share each row of a sequence of n kept tokens, up to 32 sequences: 1, 2 or 4 (at most
// p.parts), so that the longest list of a share is as short as it can be with all CTAs at work at once.
__device__ __forceinline__ int parts_of(const Moves &p, int n)
{
    const int lane = threadIdx.x & 31, seqs = gridDim.y;
    const int mine = lane < seqs ? min(max(p.num_kept[lane], 0), p.num_entries) : 0;
    const int half = (mine + 1) / 2;
    int low = 0, high = __reduce_max_sync(kFull, mine);
    while (low < high) {
        const int mid = low + (high - low) / 2;
        const int units = seqs + __popc(__ballot_sync(kFull, mine > mid)) +
                          (p.parts > 2 ? 2 * __popc(__ballot_sync(kFull, half > mid)) : 0);
        if (units <= p.units) high = mid;
        else low = mid + 1;
    }
    return n <= low ? 1 : (n + 1) / 2 <= low || p.parts == 2 ? 2 : 4;
}

template <typename C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas) compact_kernel(const Moves p)
{
    constexpr int kThreads = C::kThreads, kDepth = C::kDepth;
    // of three batches: a thread may look up the one after the next while another still writes
    // this one's rows
    __shared__ Place places[3][C::kBatch];
    __shared__ int stops[3];             // first entry that may not move, n: none
    griddep_launch_dependents();
    griddep_wait();
    const int s = blockIdx.y, tid = threadIdx.x;
    const int start = p.kept_start[s], end = p.kept_start[s + 1], n = p.num_kept[s], first = p.first[s];
    if (!(0 <= start && start <= end && end <= p.num_entries && 0 <= n && n <= end - start && first >= 0)) {
        if (blockIdx.x == 0 && tid == 0) atomicOr(p.status, PKV_DEV_BAD_LEN);
        return;
    }
    int part_chunks = p.part_chunks, batch = p.batch;
    const int part = blockIdx.x % p.parts, pair0 = blockIdx.x / p.parts * p.pairs;
    if constexpr (C::kByLength) {
        const int parts = parts_of(p, n);
        if (part >= parts) return;
        part_chunks = (p.chunks + parts - 1) / parts;
        batch = min(kThreads / part_chunks * kDepth, C::kBatch);
    }
    const int pairs = C::kPairs ? min(p.pairs, 2 * p.num_kv_heads - pair0) : 1;
    const int c0 = part * part_chunks, nc = min(part_chunks, p.chunks - c0);
    const int per_pass = kThreads / nc;              // rows of one pass of the threads
    const int c = tid % nc, k = tid / nc;
    const int32_t *row = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
    const int32_t *kept = p.kept + start;
    const int64_t limit = (int64_t)p.max_blocks_per_seq * p.block_size;
    auto place = [&](int pos) -> int64_t {
        const int id = row[pos / p.block_size];
        return id < 0 || id >= p.num_blocks
                   ? -1
                   : ((int64_t)id * p.num_kv_heads * p.block_size + pos % p.block_size) * p.chunks;
    };
    // the thread's chunk of the pool's first token
    auto chunks_of = [&](int pair) -> uint4 * {
        return (pair & 1 ? p.v_pool : p.k_pool) + c0 + c + (int64_t)(pair >> 1) * p.block_size * p.chunks;
    };
    uint4 *const base = chunks_of(pair0);
    // The list runs two batches ahead of the rows, the places one: `fetch` takes a thread's entries
    // of the batch from i0 on, `look_up` finds their places.
    constexpr int kEntries = (C::kBatch + kThreads - 1) / kThreads;
    int pos[kEntries], before[kEntries];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int j = 0; j < kEntries; ++j) {
            const int e = j * kThreads + tid, i = i0 + e;
            const bool mine = e < batch && i < n;
            pos[j] = mine ? kept[i] : 0;
            before[j] = mine && i > 0 ? kept[i - 1] : -1;
        }
    };
    auto look_up = [&](int i0, int buffer) {
#pragma unroll
        for (int j = 0; j < kEntries; ++j) {
            const int e = j * kThreads + tid, i = i0 + e;
            if (e >= batch || i >= n) continue;
            const int64_t dst = (int64_t)first + i;
            Place x = {-1, -1};
            if (pos[j] < dst || before[j] >= pos[j] || pos[j] >= limit) {
                atomicMin(&stops[buffer], i);
            } else if (pos[j] != dst) {
                x = {place(pos[j]), place((int)dst)};
                if (x.from < 0 || x.to < 0) {
                    x = {-1, -1};
                    if (blockIdx.x == 0) atomicOr(p.status, PKV_DEV_BAD_BLOCK);
                }
            }
            places[buffer][e] = x;
        }
    };
    if (tid < 3) stops[tid] = n;
    __syncthreads();
    fetch(0);
    look_up(0, 0);
    fetch(batch);
    __syncthreads();
    for (int i0 = 0, buffer = 0; i0 < n; i0 += batch, buffer = buffer == 2 ? 0 : buffer + 1) {
        const int count = min(batch, n - i0), stop = stops[buffer];
        uint4 v[kDepth];
        const int rows = k < per_pass ? min(count, stop - i0) : 0;
        // the thread's d-th chunk of the batch: where it comes from or goes to, null: nowhere
        auto chunk = [&](int d, bool source) -> uint4 * {
            int e = d * per_pass + k;
            uint4 *at = base;
            bool there = true;
            if constexpr (C::kPairs) {
                const int pair = e / batch;
                e -= pair * batch;
                at = chunks_of(pair0 + pair);
                there = pair < pairs;
            }
            if constexpr (C::kPairs) {                   // (no branch: all loads are under way at once)
                const int64_t off = source ? places[buffer][e].from : places[buffer][e].to;
                return !there || e >= rows || off < 0 ? nullptr : at + off;
            }
            if (e >= rows) return nullptr;
            const int64_t off = source ? places[buffer][e].from : places[buffer][e].to;
            return off < 0 ? nullptr : at + off;
        };
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
            if (const uint4 *from = chunk(d, true)) v[d] = *from;
        if (stop >= n) {
            look_up(i0 + batch, buffer == 2 ? 0 : buffer + 1);
            fetch(i0 + 2 * batch);
        }
        __syncthreads();                                 // every row of the batch is read
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
            if (uint4 *to = chunk(d, false)) *to = v[d];
        if (stop < n) {                                  // the same for the CTA
            if (blockIdx.x == 0 && tid == 0) atomicOr(p.status, PKV_DEV_BAD_TREE);
            return;
        }
    }
}

// Short lists: as many pairs to a CTA as fill its batch.
template <typename C>
static int launch_moves(Moves p, int parts, int num_seqs, int64_t average, cudaStream_t st)
{
    p.part_chunks = std::min((p.chunks + parts - 1) / parts, C::kThreads);
    p.parts = (p.chunks + p.part_chunks - 1) / p.part_chunks;
    const int rows = C::kThreads / p.part_chunks * C::kDepth, all = 2 * p.num_kv_heads;
    const int64_t fit = C::kPairs ? rows / std::max<int64_t>(1, average) : 1;
    p.pairs = (int32_t)std::max<int64_t>(1, std::min<int64_t>(fit, all));
    p.batch = std::min(rows / p.pairs, C::kBatch);
    const dim3 grid((unsigned)((all + p.pairs - 1) / p.pairs * p.parts), (unsigned)num_seqs);
    return launch(&compact_kernel<C>, grid, C::kThreads, st, p);
}

}  // namespace compact
}  // namespace pkv

extern "C" int kv_tree_accept(const void *tokens, const int32_t *parents, const void *targets,
                              int32_t token_bytes, const int32_t *query_start,
                              const int32_t *first, int32_t num_seqs, int32_t num_tokens,
                              int32_t *kept, int32_t *num_kept, void *next_tokens,
                              int32_t *d_status, void *stream)
{
    using namespace pkv::compact;
    if ((token_bytes != 4 && token_bytes != 8) || num_seqs < 0 || num_tokens < 0)
        return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0) return PKV_OK;
    if (!query_start || !first || !num_kept || !next_tokens || !d_status) return PKV_ERR_INVALID_ARG;
    if (num_tokens > 0 && (!tokens || !parents || !targets || !kept)) return PKV_ERR_INVALID_ARG;
    const uintptr_t wide = (uintptr_t)tokens | (uintptr_t)targets | (uintptr_t)next_tokens;
    const uintptr_t words = (uintptr_t)parents | (uintptr_t)query_start | (uintptr_t)first |
                            (uintptr_t)kept | (uintptr_t)num_kept | (uintptr_t)d_status;
    if ((wide & (uintptr_t)(token_bytes - 1)) || (words & 3u)) return PKV_ERR_INVALID_ARG;
    const Trees p = {tokens, targets, parents, query_start, first, num_seqs, num_tokens,
                     kept, num_kept, next_tokens, d_status};
    const dim3 grid((unsigned)((num_seqs + kAcceptWarps - 1) / kAcceptWarps));
    return launch(token_bytes == 8 ? &tree_accept_kernel<int64_t> : &tree_accept_kernel<int32_t>, grid,
                  32 * kAcceptWarps, (cudaStream_t)stream, p);
}

extern "C" int kv_cache_compact(const pkv_pool *pool, const int32_t *block_tables,
                                int32_t max_blocks_per_seq, const int32_t *kept,
                                const int32_t *kept_start, const int32_t *num_kept,
                                const int32_t *first, int32_t num_seqs, int32_t num_entries,
                                void *k_pool, void *v_pool, int32_t *d_status, void *stream)
{
    using namespace pkv::compact;
    pkv::PoolGeometry g;
    if (!pkv::pool_geometry(pool, &g) || !pkv::is_16bit(g)) return PKV_ERR_INVALID_ARG;
    if (num_seqs < 0 || num_entries < 0 || max_blocks_per_seq <= 0) return PKV_ERR_INVALID_ARG;
    if (g.head_dim % 8 || num_seqs > 65535 || num_entries > INT32_MAX - 8192) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_entries == 0) return PKV_OK;
    if (!block_tables || !kept || !kept_start || !num_kept || !first || !k_pool || !v_pool || !d_status)
        return PKV_ERR_INVALID_ARG;
    if (!pkv::aligned16(k_pool) || !pkv::aligned16(v_pool) || ((uintptr_t)block_tables & 3u) ||
        ((uintptr_t)kept & 3u) || ((uintptr_t)kept_start & 3u) || ((uintptr_t)num_kept & 3u) ||
        ((uintptr_t)first & 3u) || ((uintptr_t)d_status & 3u))
        return PKV_ERR_INVALID_ARG;
    Moves p = {};
    p.block_tables = block_tables;
    p.kept = kept;
    p.kept_start = kept_start;
    p.num_kept = num_kept;
    p.first = first;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_entries = num_entries;
    p.num_kv_heads = g.num_kv_heads;
    p.block_size = g.block_size;
    p.num_blocks = g.num_blocks;
    p.chunks = g.head_dim / 8;
    p.k_pool = static_cast<uint4 *>(k_pool);
    p.v_pool = static_cast<uint4 *>(v_pool);
    p.status = d_status;
    // a row is shared among CTAs where there are few, down to 64 bytes
    const int64_t ctas = (int64_t)num_seqs * g.num_kv_heads * 2, average = num_entries / num_seqs;
    const int parts = (int)std::max<int64_t>(1, std::min<int64_t>(p.chunks / 4, kMoveCtas / ctas));
    const cudaStream_t st = (cudaStream_t)stream;
    if (ctas * parts <= kFewCtas) return launch_moves<Few>(p, parts, num_seqs, average, st);
    if (average <= kBriefList) return launch_moves<Brief>(p, parts, num_seqs, average, st);
    // up to 32 long lists: as many shares of a row as their lengths ask for
    if (num_seqs <= 32 && average >= kLongList && ctas <= kManyCtas && p.chunks >= 8 &&
        p.chunks <= Many::kThreads) {
        p.parts = p.chunks >= 16 ? 4 : 2;
        p.pairs = 1;
        p.units = kManyCtas / (2 * g.num_kv_heads);
        const dim3 grid((unsigned)(2 * g.num_kv_heads * p.parts), (unsigned)num_seqs);
        return launch(&compact_kernel<Uneven>, grid, Uneven::kThreads, st, p);
    }
    return launch_moves<Many>(p, parts, num_seqs, average, st);
}
