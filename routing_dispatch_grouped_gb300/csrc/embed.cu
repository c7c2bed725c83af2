// Token embedding and its gradient.
//
// Forward:  out[t] = round(scale * table[ids[t]]).
// Backward: d_table[v] = round(scale * sum over t with ids[t] = v of dout[t]), every row written.
//   Up to 1024 tokens each block finds the tokens of its rows itself. More are sorted by id, stably,
//   so that each row's sum has one order; equal ids become runs, and a row of the table is the sum
//   of its run. Rows without a token are cleared meanwhile.
#include "moe_internal.cuh"

namespace rdg {
namespace {

template <bool IDS64>
__device__ __forceinline__ long long load_id(const void* ids, long long t) {
    return IDS64 ? static_cast<const long long*>(ids)[t]
                 : (long long)static_cast<const int*>(ids)[t];
}

// Calls f(t, id) for this thread's share of the ids, in 16-byte loads.
template <bool IDS64, typename F>
__device__ __forceinline__ void for_ids(const void* ids, int T, F f) {
    constexpr int PER = IDS64 ? 2 : 4;
    const int vectors = T / PER, tid = threadIdx.x, threads = blockDim.x;
    const uint4* p = static_cast<const uint4*>(ids);
#pragma unroll 4
    for (int i = tid; i < vectors; i += threads) {
        const uint4 u = p[i];
        if (IDS64) {
            f(2 * i, (long long)((unsigned long long)u.y << 32 | u.x));
            f(2 * i + 1, (long long)((unsigned long long)u.w << 32 | u.z));
        } else {
            f(4 * i, (long long)(int)u.x);
            f(4 * i + 1, (long long)(int)u.y);
            f(4 * i + 2, (long long)(int)u.z);
            f(4 * i + 3, (long long)(int)u.w);
        }
    }
    for (int t = vectors * PER + tid; t < T; t += threads) f(t, load_id<IDS64>(ids, t));
}
template <bool IDS64>
__device__ __forceinline__ bool any_outside(const void* ids, int T, int V) {
    bool bad = false;
    for_ids<IDS64>(ids, T, [&](int, long long id) { bad |= id < 0 || id >= V; });
    return bad;
}

__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t w, float s) {
    return pack_bf16x2(__uint_as_float(w << 16) * s, __uint_as_float(w & 0xffff0000u) * s);
}

// ---------------------------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------------------------
// A warp takes 128 16-byte vectors (2 KB) of one row: four loads a lane in flight before the first
// store, and a few tokens still spread over many SMs. Bound by memory: 16384 tokens of 5120 bf16
// values, 6600 different ones, 39.2 us, 6.1 TB/s (0.90 of the measured copy bandwidth; scattered
// rows). Eight loads a lane and streaming stores changed nothing; 2 to 6 resident blocks an SM that
// loop over the tokens were 5% slower. 64 tokens of 2880: 1.5 us, latency alone.
constexpr int kSegment = 128;

template <bool BF16, bool IDS64>
__global__ void __launch_bounds__(256)
    embed_kernel(const void* __restrict__ ids, int T, const uint4* __restrict__ table, int V,
                 int nv, int segments, float scale, uint4* __restrict__ out, bool check,
                 int* status) {
    griddep_wait();
    if (check && blockIdx.x == 0) {  // the first block (nothing waits for it) looks at all ids
        const bool bad = __syncthreads_or(any_outside<IDS64>(ids, T, V));
        if (threadIdx.x == 0) *status = bad ? MOE_ERR_DEVICE_BOUNDS : MOE_OK;
        return;
    }
    const int lane = threadIdx.x & 31;
    const long long item = ((long long)blockIdx.x - check) * 8 + (threadIdx.x >> 5);
    const long long t = item / segments;
    if (t >= T) return;
    const int c0 = (int)(item - t * segments) * kSegment + lane;
    const long long id = load_id<IDS64>(ids, t);
    const bool ok = id >= 0 && id < V;
    if (!ok && !check && lane == 0) set_status(status, MOE_ERR_DEVICE_BOUNDS);
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = c0 + 32 * i;
        v[i] = ok && c < nv ? table[id * nv + c] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = c0 + 32 * i;
        if (c >= nv) break;
        uint4 u = v[i];
        if (BF16) {
            u = make_uint4(scale_bf16x2(u.x, scale), scale_bf16x2(u.y, scale),
                           scale_bf16x2(u.z, scale), scale_bf16x2(u.w, scale));
        } else {
            u = make_uint4(__float_as_uint(__uint_as_float(u.x) * scale),
                           __float_as_uint(__uint_as_float(u.y) * scale),
                           __float_as_uint(__uint_as_float(u.z) * scale),
                           __float_as_uint(__uint_as_float(u.w) * scale));
        }
        if (!ok) u = make_uint4(0, 0, 0, 0);  // not scale * 0: the scale may be infinite
        out[t * nv + c] = u;
    }
}

constexpr int kTile = 1024;              // tokens a block sorts in shared memory
constexpr int kRuns = 16;                // runs a round merges into one
constexpr uint32_t kNoToken = 1u << 31;  // the key of an id outside [0, V): after every id

// How many of the n sorted keys are below k (or not above it, with `equal`). `top` is a power of
// two that is at least n.
__device__ __forceinline__ int count_below(const uint32_t* keys, int n, int top, uint32_t k,
                                           bool equal) {
    int pos = 0;
    for (int step = top; step > 0; step >>= 1) {
        const int at = pos + step;
        if (at <= n) {
            const uint32_t x = keys[at - 1];
            if (x < k || (equal && x == k)) pos = at;
        }
    }
    return pos;
}

template <bool BF16>
struct Row;
template <>
struct Row<true> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void add(uint4 u, float* a) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[2 * i] += __uint_as_float(w[i] << 16);
            a[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Row<false> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void add(uint4 u, float* a) {
        a[0] += __uint_as_float(u.x);
        a[1] += __uint_as_float(u.y);
        a[2] += __uint_as_float(u.z);
        a[3] += __uint_as_float(u.w);
    }
};

template <int N, bool OUT_BF16>
__device__ __forceinline__ void store_row(void* out, size_t at, const float* a, float scale) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
        if (OUT_BF16)
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at + j) =
                make_uint2(pack_bf16x2(a[j] * scale, a[j + 1] * scale),
                           pack_bf16x2(a[j + 2] * scale, a[j + 3] * scale));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(out) + at + j) =
                make_float4(a[j] * scale, a[j + 1] * scale, a[j + 2] * scale, a[j + 3] * scale);
    }
}

__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
                 "r"(bytes)
                 : "memory");
}

// Rows of the table that no token has are cleared by bulk copies of zeros from shared memory (one
// instruction for up to 8 KB), or, where a row is no multiple of 16 bytes (bf16 rows of fp32
// gradients), by 8-byte stores.
constexpr int kZeroBytes = 8192;
constexpr int kMaxClearRows = 1024;  // of one block

// Rows of the table for a block that clears them: 64 KB or more (with 32 KB the clearing of 262 MB
// took 52 us, with 64 KB and 128 KB 43 to 44, with 256 KB 46), and more for many tokens, since each
// such block reads all ids.
int rows_to_clear(long long row_bytes, int T) {
    int rows = 1;
    while (rows < kMaxClearRows && (rows * row_bytes < 65536 || (long long)rows * 1024 < T))
        rows *= 2;
    return rows;
}

__device__ __forceinline__ void zero_fill(uint4* zeros) {
    for (int i = threadIdx.x; i < kZeroBytes / 16; i += blockDim.x)
        zeros[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();  // the bulk copies read what was written here
}
// Starts the clearing of the rows [0, n) from `first` on whose mark is 0; the caller waits with
// bulk_wait_read<0>() before it leaves. Small rows go several to a copy.
__device__ __forceinline__ void clear_unmarked(uint8_t* first, const uint8_t* marks, int n,
                                               long long row_bytes, const uint4* zeros) {
    const int tid = threadIdx.x, threads = blockDim.x;
    if (row_bytes % 16 == 0) {
        const int group = row_bytes < kZeroBytes ? (int)(kZeroBytes / row_bytes) : 1;
        for (int r = tid; r < n; r += threads) {
            if (marks[r] || (r % group != 0 && !marks[r - 1])) continue;  // none, or not the first
            int end = r + 1;
            while (end < n && end % group != 0 && !marks[end]) ++end;
            uint8_t* row = first + r * row_bytes;
            const long long bytes = (end - r) * row_bytes;
            for (long long b = 0; b < bytes; b += kZeroBytes)
                bulk_store(row + b, smem_u32(zeros),
                           (uint32_t)(bytes - b < kZeroBytes ? bytes - b : kZeroBytes));
        }
        bulk_commit();
    } else {
        const int width = (int)(row_bytes / 8);
        for (int r = tid >> 5; r < n; r += threads / 32) {
            if (marks[r]) continue;
            uint2* row = reinterpret_cast<uint2*>(first + r * row_bytes);
            for (int c = tid & 31; c < width; c += 32) row[c] = make_uint2(0, 0);
        }
    }
}

// ---------------------------------------------------------------------------------------------
// few tokens: one kernel
// ---------------------------------------------------------------------------------------------
// A block takes some rows of the table: it reads all ids, keeps the tokens of its rows in ascending
// order, starts the clearing of the rows without one and sums the others. Where a row has fewer
// vectors than the block threads, groups of threads take consecutive parts of its tokens, which
// are then added in order. Blocks along y share a row's columns. Bound by memory, by the clearing:
// 1000 tokens into 32000 rows of 8 KB 43 us, 6.2 TB/s (0.91 of the measured copy bandwidth); by
// sort, sums and join 49.8.
constexpr int kFewChunks = kEmbedFewTokens / 32;
static_assert(kFewChunks == 32, "a lane of one warp adds each chunk's count");

template <int kFewThreads, bool BF16, bool OUT_BF16, bool IDS64>
__global__ void __launch_bounds__(kFewThreads, 1024 / kFewThreads)
    embed_few_kernel(const uint4* __restrict__ dout, const void* __restrict__ ids, int T, int V,
                     int nv, int rows_of_block, float scale, void* out, long long row_bytes,
                     int* status) {
    constexpr int N = Row<BF16>::N, AHEAD = 8, kFewWarps = kFewThreads / 32;
    __shared__ uint8_t has[kMaxClearRows];
    __shared__ __align__(128) uint4 zeros[kZeroBytes / 16];
    __shared__ int16_t row_of[kEmbedFewTokens];  // row of each token, or -1
    __shared__ int16_t list[kEmbedFewTokens];    // the tokens of one row
    __shared__ int before[kFewChunks + 1];
    __shared__ __align__(16) float part[kFewThreads * N];
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long v0 = (long long)blockIdx.x * rows_of_block;
    zero_fill(zeros);
    for (int r = tid; r < rows_of_block; r += kFewThreads) has[r] = 0;
    __syncthreads();
    bool bad = false;
    for (int t = tid; t < T; t += kFewThreads) {
        const long long id = load_id<IDS64>(ids, t), r = id - v0;
        bad |= id < 0 || id >= V;
        const bool mine = id < V && r >= 0 && r < rows_of_block;
        row_of[t] = mine ? (int16_t)r : (int16_t)-1;
        if (mine) has[r] = 1;
    }
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0)
        *status = bad ? MOE_ERR_DEVICE_BOUNDS : MOE_OK;
    const int rows = (int)(V - v0 < rows_of_block ? V - v0 : rows_of_block);
    if (blockIdx.y == 0)
        clear_unmarked(static_cast<uint8_t*>(out) + v0 * row_bytes, has, rows, row_bytes, zeros);
    // this block's vectors of each row: [first, first + width)
    const int share = (nv + (int)gridDim.y - 1) / (int)gridDim.y, first = (int)blockIdx.y * share;
    const int width = nv - first < share ? nv - first : share;
    if (width <= 0) return;
    const int parts = width < kFewThreads ? kFewThreads / width : 1;
    int r = -1;
    for (;;) {
        // the next row that has a token
        const int from = r + 1;
        r = rows;
        for (int b = from; b < rows; b += 32) {
            const unsigned m = __ballot_sync(0xffffffffu, b + lane < rows && has[b + lane]);
            if (m) {
                r = b + __ffs(m) - 1;
                break;
            }
        }
        if (r >= rows) break;
        // this row's tokens, ascending: counts of each 32, their running sums, places
        unsigned mask[(kFewChunks + kFewWarps - 1) / kFewWarps];
#pragma unroll
        for (int i = 0; i < (kFewChunks + kFewWarps - 1) / kFewWarps; ++i) {
            const int t = (i * kFewWarps + warp) * 32 + lane;
            mask[i] = __ballot_sync(0xffffffffu, t < T && row_of[t] == r);
            if (lane == 0) before[i * kFewWarps + warp] = __popc(mask[i]);
        }
        __syncthreads();
        if (warp == 0) {
            const int own = before[lane];  // kFewChunks == 32
            int sum = own;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int x = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += x;
            }
            before[lane] = sum - own;
            if (lane == 31) before[kFewChunks] = sum;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < (kFewChunks + kFewWarps - 1) / kFewWarps; ++i)
            if (mask[i] >> lane & 1)
                list[before[i * kFewWarps + warp] + __popc(mask[i] & ((1u << lane) - 1))] =
                    (int16_t)((i * kFewWarps + warp) * 32 + lane);
        __syncthreads();
        const int n = before[kFewChunks];
        const int group = parts > 1 ? tid / width : 0;
        int each = (n + parts - 1) / parts;  // tokens a group; up to 32 are summed as they stand
        if (each < 32) each = 32;
        const int lo = group * each < n ? group * each : n, hi = lo + each < n ? lo + each : n;
        const size_t row = (size_t)(v0 + r) * nv + first;  // in vectors
        for (int c = tid - group * width; c < width && group < parts; c += kFewThreads) {
            float acc[N];
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = 0.f;
            for (int i0 = lo; i0 < hi; i0 += AHEAD) {
                uint4 u[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    if (i0 + i < hi) u[i] = dout[(size_t)list[i0 + i] * nv + first + c];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    if (i0 + i < hi) Row<BF16>::add(u[i], acc);
            }
            if (parts == 1)
                store_row<N, OUT_BF16>(out, (row + c) * N, acc, scale);
            else
#pragma unroll
                for (int j = 0; j < N; ++j) part[tid * N + j] = acc[j];
        }
        if (parts > 1) {
            __syncthreads();
            if (tid < width) {
                float acc[N];
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] = part[tid * N + j];
                for (int g = 1; g < parts; ++g)
#pragma unroll
                    for (int j = 0; j < N; ++j) acc[j] += part[(g * width + tid) * N + j];
                store_row<N, OUT_BF16>(out, (row + tid) * N, acc, scale);
            }
        }
        __syncthreads();  // the next row writes before[], list[] and part[] again
    }
    bulk_wait_read<0>();
}

// ---------------------------------------------------------------------------------------------
// more tokens: sorted by id
// ---------------------------------------------------------------------------------------------
struct ClearArgs {
    const void* ids;
    uint8_t* out;
    long long row_bytes;
    int T, V, rows;
    int* status;
};

// Clears the rows [block * rows, ...) that no token has: the block marks those that its pass over
// the ids meets. Nothing of this waits for the sort, beside which it runs. Block 0 writes the
// status word, since it sees all ids.
template <bool IDS64>
__device__ void clear_rows(const ClearArgs& a, int block) {
    __shared__ uint8_t has[kMaxClearRows];
    __shared__ __align__(128) uint4 zeros[kZeroBytes / 16];
    const int tid = threadIdx.x, threads = blockDim.x;
    const long long v0 = (long long)block * a.rows;
    for (int i = tid; i < a.rows; i += threads) has[i] = 0;
    zero_fill(zeros);
    __syncthreads();
    bool bad = false;
    for_ids<IDS64>(a.ids, a.T, [&](int, long long id) {
        const long long r = id - v0;
        bad |= id < 0 || id >= a.V;
        if (r >= 0 && r < a.rows) has[r] = 1;
    });
    bad = __syncthreads_or(bad);
    if (block == 0 && tid == 0) *a.status = bad ? MOE_ERR_DEVICE_BOUNDS : MOE_OK;
    clear_unmarked(a.out + v0 * a.row_bytes, has, (int)(v0 + a.rows > a.V ? a.V - v0 : a.rows),
                   a.row_bytes, zeros);
    bulk_wait_read<0>();
}

// Blocks [0, tiles): a tile of 1024 tokens each. Each warp ranks its 32 by comparing all pairs,
// then runs are merged two by two: an element's place is its own rank plus its rank in the other
// run (found by bisection; on equal ids the left run comes first, which keeps the order of the
// tokens). The blocks after those clear rows of the table: 1.27 GB of zeros in 176 us, as fast as
// memory takes them, and the sort within that time.
template <bool IDS64>
__global__ void __launch_bounds__(kTile)
    embed_sort_kernel(const void* __restrict__ ids, int T, int V, uint32_t* __restrict__ keys,
                      int* __restrict__ tokens, int tiles, const ClearArgs clear) {
    __shared__ uint32_t ks[2][kTile];
    __shared__ short is[2][kTile];
    griddep_wait();
    if ((int)blockIdx.x >= tiles) {
        clear_rows<IDS64>(clear, (int)blockIdx.x - tiles);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31;
    const long long t0 = (long long)blockIdx.x * kTile, t = t0 + tid;
    uint32_t k = kNoToken;
    if (t < T) {
        const long long id = load_id<IDS64>(ids, t);
        if (id >= 0 && id < V) k = (uint32_t)id;
    }
    int rank = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const uint32_t x = __shfl_sync(0xffffffffu, k, j);
        rank += x < k || (x == k && j < lane);
    }
    ks[0][(tid & ~31) + rank] = k;
    is[0][(tid & ~31) + rank] = (short)tid;
    __syncthreads();
    int cur = 0;
    for (int run = 32; run < kTile; run *= 2) {
        const uint32_t x = ks[cur][tid];
        const int base = tid & ~(2 * run - 1);
        const bool right = (tid & run) != 0;
        const int other = base + (right ? 0 : run);
        const int to = base + (tid & (run - 1)) + count_below(ks[cur] + other, run, run, x, right);
        ks[cur ^ 1][to] = x;
        is[cur ^ 1][to] = is[cur][tid];
        cur ^= 1;
        __syncthreads();
    }
    if (t < T) {  // the places past the end come last: their keys are the largest, their order too
        keys[t] = ks[cur][tid];
        tokens[t] = (int)(t0 + is[cur][tid]);
    }
}

// Up to 8192 tokens: a token's place is the number of tokens with a lower id and of those before it
// with its own, counted. A block places 32 tokens, its eight warps count an eighth of the keys each
// (broadcast loads of four). T^2 comparisons, so not for long inputs: 4096 tokens of 184 columns
// took 24 us in all with the sort and a merge in place of this kernel, 14 with it. The blocks
// after those clear rows of the table.
constexpr int kCountThreads = 256;
template <bool IDS64>
__global__ void __launch_bounds__(kCountThreads)
    embed_count_kernel(const void* __restrict__ ids, int T, int V, uint32_t* __restrict__ keys,
                       int* __restrict__ tokens, int blocks, const ClearArgs clear) {
    __shared__ __align__(16) uint32_t ks[kEmbedCountTokens];
    __shared__ int counts[kCountThreads];
    griddep_wait();
    if ((int)blockIdx.x >= blocks) {
        clear_rows<IDS64>(clear, (int)blockIdx.x - blocks);
        return;
    }
    for_ids<IDS64>(ids, T, [&](int t, long long id) {
        ks[t] = id >= 0 && id < V ? (uint32_t)id : kNoToken;
    });
    const int vectors = (T + 3) / 4;
    for (int t = T + threadIdx.x; t < 4 * vectors; t += kCountThreads) ks[t] = ~0u;
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e0 = blockIdx.x * 32, e = e0 + lane;
    const uint32_t k = e < T ? ks[e] : 0u;
    const uint4* kv = reinterpret_cast<const uint4*>(ks);
    int n = 0;
    // before the block's own 32 tokens ids up to k count, after them ids below k
    auto count = [&](int from, int to, uint32_t limit) {
#pragma unroll 8
        for (int i = from + warp; i < to; i += kCountThreads / 32) {
            const uint4 x = kv[i];
            n += (x.x < limit) + (x.y < limit) + (x.z < limit) + (x.w < limit);
        }
    };
    count(0, e0 / 4, k + 1);
    count(e0 / 4 + 8, vectors, k);
    for (int t = e0 + warp; t < e0 + 32 && t < T; t += kCountThreads / 32)
        n += ks[t] < k + (t < e ? 1u : 0u);
    counts[threadIdx.x] = n;
    __syncthreads();
    if (warp == 0 && e < T) {
#pragma unroll
        for (int w = 1; w < kCountThreads / 32; ++w) n += counts[w * 32 + lane];
        keys[n] = k;
        tokens[n] = e;
    }
}

// Up to 16 sorted runs of `run` tokens each (a power of two) become one: an element's place is its
// own rank plus its rank in each of the other runs. Four threads take an element, four runs each;
// their bisections go step by step together, so that loads overlap. (16384 tokens: one bisection
// after the other took 34 us, 16 in step by one thread 13.)
constexpr int kMergeThreads = 256, kMergeShare = 4;
__global__ void __launch_bounds__(kMergeThreads)
    embed_merge_kernel(const uint32_t* __restrict__ keys, const int* __restrict__ tokens, int T,
                       int run, uint32_t* __restrict__ keys_out, int* __restrict__ tokens_out) {
    constexpr int kMine = kRuns / kMergeShare;
    griddep_wait();
    const long long e = ((long long)blockIdx.x * kMergeThreads + threadIdx.x) / kMergeShare;
    const int share = threadIdx.x % kMergeShare;
    const long long at_e = e < T ? e : T - 1;  // threads past the end go along for the shuffles
    const uint32_t k = keys[at_e];
    const int mine = (int)(at_e / run), first = mine / kRuns * kRuns, own = share * kMine + first;
    int n[kMine], pos[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        const long long left = T - (long long)(own + j) * run;
        n[j] = own + j == mine || left <= 0 ? 0 : (int)(left < run ? left : run);
        pos[j] = 0;
    }
    for (int step = run; step > 0; step >>= 1) {
        uint32_t x[kMine];
#pragma unroll
        for (int j = 0; j < kMine; ++j) {  // past the run's end: any key, not used
            const int at = pos[j] + step;
            x[j] = keys[at <= n[j] ? (long long)(own + j) * run + at - 1 : 0];
        }
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int at = pos[j] + step;
            const bool below = x[j] < k || (own + j < mine && x[j] == k);
            pos[j] = at <= n[j] && below ? at : pos[j];
        }
    }
    int rank = 0;
#pragma unroll
    for (int j = 0; j < kMine; ++j) rank += pos[j];
#pragma unroll
    for (int o = 1; o < kMergeShare; o *= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (share == 0 && e < T) {
        const long long to = (long long)first * run + (e - (long long)mine * run) + rank;
        keys_out[to] = k;
        tokens_out[to] = tokens[e];
    }
}

// ---------------------------------------------------------------------------------------------
// sums over the runs of equal ids
// ---------------------------------------------------------------------------------------------
constexpr int kSumThreads = 128;  // a block takes 128 vectors of dout's rows (a slice)
constexpr int kMaxChunk = 512;

struct SumArgs {
    const uint4* dout;
    const uint32_t* keys;  // sorted
    const int* tokens;
    void* out;             // [V, d]
    float* part;           // [chunks, 2, d]
    int T, d, nv, chunk, chunks, slices;
    float scale;
};

// A block takes a chunk of the sorted tokens and a slice of the columns. A run that lies within
// the chunk is finished here; of a run that goes on in another chunk the sum of this chunk's part
// is kept (place 0: it began before the chunk; 1: it begins here). Bound by memory: 37 us for 16384
// rows of 10 KB into 6600 (0.95 of the measured copy bandwidth). Eight rows are on their way at
// a time: with 16, registers left fewer blocks resident (43 us instead of 37 for 16384 rows).
template <bool BF16, bool OUT_BF16>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const SumArgs a) {
    constexpr int N = Row<BF16>::N, AHEAD = 8;
    __shared__ uint32_t ks[kMaxChunk + 2];
    __shared__ int ts[kMaxChunk];
    griddep_wait();
    const int tid = threadIdx.x;
    const int chunk = (int)(blockIdx.x / a.slices), slice = (int)(blockIdx.x % a.slices);
    const long long e0 = (long long)chunk * a.chunk;
    const int n = (int)(a.T - e0 < a.chunk ? a.T - e0 : a.chunk);
    for (int i = tid; i < n + 2; i += kSumThreads) {  // with a neighbour on each side
        const long long e = e0 + i - 1;
        ks[i] = e >= 0 && e < a.T ? a.keys[e] : kNoToken;
    }
    for (int i = tid; i < n; i += kSumThreads) ts[i] = a.tokens[e0 + i];
    __syncthreads();
    const int c = slice * kSumThreads + tid;
    if (c >= a.nv) return;
    const bool head = ks[0] == ks[1], tail = ks[n] == ks[n + 1];
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.f;
    bool from_before = head;
    for (int i0 = 0; i0 < n; i0 += AHEAD) {
        uint4 u[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (i0 + i < n && ks[i0 + i + 1] != kNoToken)
                u[i] = a.dout[(size_t)ts[i0 + i] * a.nv + c];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int e = i0 + i;
            if (e >= n) break;
            const uint32_t k = ks[e + 1];
            if (k == kNoToken) return;  // those come last
            Row<BF16>::add(u[i], acc);
            if (e + 1 < n && ks[e + 2] == k) continue;
            const bool goes_on = e + 1 == n && tail;
            if (from_before || goes_on) {
                float* part = a.part + ((size_t)chunk * 2 + (from_before ? 0 : 1)) * a.d + c * N;
#pragma unroll
                for (int j = 0; j < N; j += 4)
                    *reinterpret_cast<float4*>(part + j) =
                        make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
            } else {
                store_row<N, OUT_BF16>(a.out, (size_t)k * a.d + (size_t)c * N, acc, a.scale);
            }
            from_before = false;
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = 0.f;
        }
    }
}

// Runs over several chunks: the block of the chunk in which such a run begins adds its parts. Four
// columns a thread; four groups of threads take consecutive parts, and their sums are added in
// order. Latency, 5 to 10 us: most blocks find no such run.
constexpr int kJoinColumns = 128, kJoinGroups = 4;  // threads along the columns; groups
template <bool OUT_BF16>
__global__ void __launch_bounds__(kJoinColumns * kJoinGroups) embed_join_kernel(const SumArgs a) {
    __shared__ float4 sums[kJoinGroups][kJoinColumns];
    griddep_wait();
    const int j = blockIdx.x, x = threadIdx.x % kJoinColumns, group = threadIdx.x / kJoinColumns;
    const int c = (blockIdx.y * kJoinColumns + x) * 4;
    const long long first = (long long)j * a.chunk, next = first + a.chunk;
    const uint32_t k = a.keys[next];  // next < T: j is not the last chunk
    const uint32_t last_of_mine = a.keys[next - 1];
    const uint32_t before = first > 0 ? a.keys[first - 1] : kNoToken;
    if (k == kNoToken || last_of_mine != k || before == k) return;
    int parts = 1;  // this chunk, and those after it whose first token has the run's id
    for (int from = j + 1; from < a.chunks; from += kJoinColumns * kJoinGroups) {
        const int i = from + threadIdx.x;
        const int n = __syncthreads_count(i < a.chunks && a.keys[(long long)i * a.chunk] == k);
        parts += n;
        if (n < kJoinColumns * kJoinGroups) break;
    }
    const int lo = (int)((long long)parts * group / kJoinGroups);
    const int hi = (int)((long long)parts * (group + 1) / kJoinGroups);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < a.d) {
#pragma unroll 8
        for (int i = lo; i < hi; ++i) {
            const size_t at = (size_t)(j + i) * 2 + (i == 0 ? 1 : 0);
            const float4 v = *reinterpret_cast<const float4*>(a.part + at * a.d + c);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
    }
    sums[group][x] = s;
    __syncthreads();
    if (group != 0 || c >= a.d) return;
#pragma unroll
    for (int g = 1; g < kJoinGroups; ++g) {
        const float4 v = sums[g][x];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    const float acc[4] = {s.x, s.y, s.z, s.w};
    store_row<4, OUT_BF16>(a.out, (size_t)k * a.d + c, acc, a.scale);
}

// Sorted tokens that a block sums. Long chunks leave fewer runs to join, short ones more blocks:
// of 16, 32, ... 512 the longest with which the blocks still fill the SMs eight deep (16384 tokens
// of 5120 columns: 16 took 247 us, 32 239, 64 235; 8471 of 104: 19.2, 21.4 and 25.0), or the
// shortest that leaves at most 1024 chunks, whichever is longer. Past 524288 tokens chunks stay at
// 512, and a run over all tokens is joined from T / 512 parts, a quarter of them by each group of
// threads one after the other.
// A GB300's SMs as a number: the workspace's size goes by the chunks and must not change with the
// device that is current.
constexpr int kChunkSms = 152;
int chunk_of(int T, int d) {
    const long long slices = (d + 1023) / 1024;
    int c = 16;
    while (c < kMaxChunk && (T / (2 * c) * slices >= 8 * kChunkSms || (long long)c * 1024 < T))
        c *= 2;
    return c;
}

template <int THREADS>
auto few_kernel(bool bf16, bool out_bf16, bool ids64) {
    if (ids64)
        return bf16 ? (out_bf16 ? embed_few_kernel<THREADS, true, true, true>
                                : embed_few_kernel<THREADS, true, false, true>)
                    : (out_bf16 ? embed_few_kernel<THREADS, false, true, true>
                                : embed_few_kernel<THREADS, false, false, true>);
    return bf16 ? (out_bf16 ? embed_few_kernel<THREADS, true, true, false>
                            : embed_few_kernel<THREADS, true, false, false>)
                : (out_bf16 ? embed_few_kernel<THREADS, false, true, false>
                            : embed_few_kernel<THREADS, false, false, false>);
}

}  // namespace

size_t embed_backward_scratch_bytes(int T, int d) {
    const size_t chunk = chunk_of(T, d), chunks = (T + chunk - 1) / chunk;
    return 4 * (((size_t)T * 4 + 255) / 256 * 256) + chunks * 2 * d * 4;
}

cudaError_t launch_embed(const void* ids, bool ids64, int T, const void* table, bool bf16, int V,
                         int d, float scale, void* out, int* status, cudaStream_t s) {
    const int nv = d / (bf16 ? 8 : 4), segments = (nv + kSegment - 1) / kSegment;
    const bool check = status && T <= kEmbedCheckTokens;  // else the word was cleared before
    const long long blocks = ((long long)T * segments + 7) / 8 + (check ? 1 : 0);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    auto fn = bf16 ? (ids64 ? embed_kernel<true, true> : embed_kernel<true, false>)
                   : (ids64 ? embed_kernel<false, true> : embed_kernel<false, false>);
    return launch_kernel(fn, dim3((unsigned)blocks), dim3(256), 0, s, ids, T,
                         static_cast<const uint4*>(table), V, nv, segments, scale,
                         static_cast<uint4*>(out), check, status);
}

cudaError_t launch_embed_backward(const void* dout, const void* ids, bool ids64, bool bf16, int T,
                                  int d, int V, float scale, bool out_bf16, void* d_table,
                                  void* scratch, int* status, cudaStream_t s) {
    const long long row_bytes = (long long)d * (out_bf16 ? 2 : 4);
    const int nv = d / (bf16 ? 8 : 4);
    int rows = rows_to_clear(row_bytes, T);
    if (T <= kEmbedFewTokens) {
        // a block sums its rows one after the other: not many with a token in one block
        while (rows > 8 && (long long)rows * T > 16ll * V) rows /= 2;
        // Rows of up to 256 vectors take blocks of 256 threads, wider ones of 512: 43 and 45 us for
        // 1000 rows of 256, 67 and 55 us for 509 of 1280.
        const int threads = nv > 256 ? 512 : 256;
        const auto fn = threads == 256 ? few_kernel<256>(bf16, out_bf16, ids64)
                                       : few_kernel<512>(bf16, out_bf16, ids64);
        const long long blocks = ((long long)V + rows - 1) / rows;
        int slices = 1;  // of the columns, where the rows alone are too few blocks
        while (blocks * slices < 4 * device_sm_count() && nv > 64 * slices) slices *= 2;
        return launch_kernel(fn, dim3((unsigned)blocks, slices), dim3(threads), 0, s,
                             static_cast<const uint4*>(dout), ids, T, V, nv, rows, scale, d_table,
                             row_bytes, status);
    }
    uint8_t* w = static_cast<uint8_t*>(scratch);
    const size_t words = ((size_t)T * 4 + 255) / 256 * 256;
    uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(w), reinterpret_cast<uint32_t*>(w + words)};
    int* tokens[2] = {reinterpret_cast<int*>(w + 2 * words), reinterpret_cast<int*>(w + 3 * words)};

    const ClearArgs c = {ids, static_cast<uint8_t*>(d_table), row_bytes, T, V, rows, status};
    const long long clears = ((long long)V + rows - 1) / rows;
    const bool count = T <= kEmbedCountTokens;
    const int sorts = count ? (T + 31) / 32 : (int)(((long long)T + kTile - 1) / kTile);
    if (sorts + clears > 0x7fffffffll) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)(sorts + clears));
    cudaError_t e =
        count ? launch_kernel(ids64 ? embed_count_kernel<true> : embed_count_kernel<false>, grid,
                              dim3(kCountThreads), 0, s, ids, T, V, keys[0], tokens[0], sorts, c)
              : launch_kernel(ids64 ? embed_sort_kernel<true> : embed_sort_kernel<false>, grid,
                              dim3(kTile), 0, s, ids, T, V, keys[0], tokens[0], sorts, c);
    int cur = 0;
    PdlScope pdl(true);
    for (long long run = kTile; !count && run < T && e == cudaSuccess; run *= kRuns, cur ^= 1)
        e = launch_kernel(embed_merge_kernel,
                          dim3((unsigned)(((long long)T * kMergeShare + kMergeThreads - 1) / kMergeThreads)),
                          dim3(kMergeThreads), 0, s, (const uint32_t*)keys[cur],
                          (const int*)tokens[cur], T, (int)run, keys[cur ^ 1], tokens[cur ^ 1]);
    if (e != cudaSuccess) return e;
    SumArgs a;
    a.dout = static_cast<const uint4*>(dout);
    a.keys = keys[cur];
    a.tokens = tokens[cur];
    a.out = d_table;
    a.part = reinterpret_cast<float*>(w + 4 * words);
    a.T = T;
    a.d = d;
    a.nv = nv;
    a.chunk = chunk_of(T, d);
    a.chunks = (int)(((long long)T + a.chunk - 1) / a.chunk);
    a.slices = (nv + kSumThreads - 1) / kSumThreads;
    a.scale = scale;
    const long long blocks = (long long)a.chunks * a.slices;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    auto sum = bf16 ? (out_bf16 ? embed_sum_kernel<true, true> : embed_sum_kernel<true, false>)
                    : (out_bf16 ? embed_sum_kernel<false, true> : embed_sum_kernel<false, false>);
    e = launch_kernel(sum, dim3((unsigned)blocks), dim3(kSumThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    auto join = out_bf16 ? embed_join_kernel<true> : embed_join_kernel<false>;
    return launch_kernel(join, dim3(a.chunks - 1, (d + 4 * kJoinColumns - 1) / (4 * kJoinColumns)),
                         dim3(kJoinColumns * kJoinGroups), 0, s, a);
}

}  // namespace rdg
