// get_rows.cu -- embedding lookup from a plain or block-quantised table, and
// the gradient of the table.
//
//   y[m, t]  = scale * W[m, ids[t]]
//   dW[m, v] = scale * sum over the t with ids[t] == v of dy[m, t]
//
// (ggml's GET_ROWS and GET_ROWS_BACK; the latter is among the training
// operations that "metal: OUT_PROD runs batched, broadcast and narrow shapes
// on the GPU" lists as still running on the CPU.)
#include <cooperative_groups.h>

#include <algorithm>

#include "oop_internal.cuh"
#include "quant.cuh"
#include "rows.cuh"

namespace cg = cooperative_groups;

namespace oop {
namespace {

constexpr int kThreads = 256;

// Bound by memory: a row is read and written once.  A CTA takes R tokens and
// kThreads * E columns of their rows; every load is issued before the first
// store, so a CTA waits for memory twice (the ids, then all of its rows).  bf16,
// 16384 tokens x 4096: 33 us, 8.1 TB/s of rows, of which the frequent ones come
// from L2 (one token per CTA and scalar loads: 92 us); q8_0, 8192 x 4096 to f32:
// 34.6 us, 72% of the measured copy rate, decoding four elements per thread, one token
// per CTA.  The other block types to bf16, same sizes: 31 (q4_0) to 41 us (q5_1), and 49
// (q2_K) to 74 us (q3_K), 41% to 16%: the codes are read by single bytes and a
// block's scale is found again for every element.
template <int TYPE, int OUT, int E, int R>
__global__ void __launch_bounds__(kThreads) get_rows_kernel(const void *table, int64_t nb_table,
                                                            const int32_t *ids, void *dst,
                                                            int64_t nb_dst, int64_t M, int64_t V,
                                                            int64_t T, float scale, int *status) {
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * R;
    const int64_t m = (static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x) * E;
    int32_t id[R];
#pragma unroll
    for (int r = 0; r < R; ++r) id[r] = t0 + r < T ? ids[t0 + r] : -1;
    if (m >= M) return;
    float v[R][E];
    if constexpr (is_plain_type<TYPE>()) {
        Packed<TYPE, E> raw[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            raw[r].raw = {};
            if (id[r] >= 0 && id[r] < V)
                raw[r] = load_packed<TYPE, E>(row_of<TYPE>(table, nb_table, id[r]) + m);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) raw[r].get(v[r]);
    } else {
        using F = QFormat<TYPE>;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = id[r] >= 0 && id[r] < V;
            const uint8_t *blk = static_cast<const uint8_t *>(table) +
                                 (in ? id[r] : 0) * nb_table + m / F::QK * F::BYTES;
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[r][e] = in ? decode<TYPE>(blk, static_cast<int>(m % F::QK) + e) : 0.f;
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (t0 + r >= T) break;
        const bool in = id[r] >= 0 && id[r] < V;
        if (m == 0 && !in) record_status(status, OOP_ERR_BAD_ID);
        const float by = in ? scale : 0.f;             // (0 times an infinite scale is none)
#pragma unroll
        for (int e = 0; e < E; ++e) v[r][e] *= by;
        store_stream<OUT, E>(row_of<OUT>(dst, nb_dst, t0 + r) + m, v[r]);
    }
}

// ---- the gradient ---------------------------------------------------------
//
// The (id, t) pairs are sorted by id, equal ids in ascending t, by a stable
// radix sort in one cluster of 8 CTAs, while the other SMs write the table's
// zeros (a launch that starts with the sort): the zeros are most of the work,
// and the sort hides behind them.  The sorted list is then cut into chunks of
// kChunk tokens, however the ids fall, so a token that fills half the batch is
// spread like any other: a CTA adds up the rows of its chunk, run by run,
// writes the sum of a run that lies inside it to the table and the sum of a
// run that crosses its ends to the workspace, where a last launch joins the
// parts of each such run in a fixed order.  Each launch is on its way while the
// one before drains.
//
// f32, 8192 tokens x 2560 into 50257 rows: 97 us, 91% of the measured copy rate;
// the zeros take 68 us (the sort's 14 hidden behind them), the sums 24 and the
// join 6.  Where there are few zeros to write, the sort is the longest part.

constexpr int kSortCluster = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBits = 9;                        // of the id, sorted in one pass
constexpr int kMaxBins = 1 << kMaxBits;
constexpr int kRanked = 1024;                      // tokens sorted by counting: an eighth per CTA, 8 threads each
static_assert(kRanked / kSortCluster * 8 <= kSortThreads);
constexpr int kSortSmem = (kSortWarps * kMaxBins + 2 * kMaxBins + 32) * 4;

struct SortPlan {
    int bits, passes;                              // bits of one pass
};

// Keys are 0 .. V (V: an id outside the table, sorted last).
SortPlan sort_plan(int64_t V) {
    int n = 1;
    while ((V >> n) != 0) ++n;
    SortPlan p;
    p.passes = (n + kMaxBits - 1) / kMaxBits;
    p.bits = (n + p.passes - 1) / p.passes;
    return p;
}

struct SortArgs {
    const int32_t *ids;
    uint2 *buf[2];                                 // (key, t), written in turn; the last pass writes buf[0]
    uint2 *crossing;                               // runs in several chunks: (first, last chunk)
    int *n_crossing;
    int64_t T, V;
    int bits, passes;
    int *status;
};

constexpr int kChunk = 32;                         // sorted tokens per CTA of the sums

// Zeros, 32 bytes per thread and as many CTAs as that takes: 7.2 TB/s, where
// loops over the same range by one to sixteen CTAs per SM reach 6.1 to 6.6.
__global__ void __launch_bounds__(kThreads) fill_zero_kernel(float *p, int64_t n) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t head = min(n, static_cast<int64_t>((32 - (reinterpret_cast<uintptr_t>(p) & 31)) & 31) / 4);
    const int64_t eights = (n - head) / 8, tail = head + eights * 8;
    if (i < eights)
        asm volatile("st.global.v8.f32 [%0], {%1, %1, %1, %1, %1, %1, %1, %1};" ::"l"(p + head + 8 * i),
                     "f"(0.f) : "memory");
    if (i < head) p[i] = 0.f;
    if (i < n - tail) p[tail + i] = 0.f;
    let_next_start();
    // this grid must not end before the sort it started beside
    if (blockIdx.x == gridDim.x - 1) wait_previous();
}

__global__ void __launch_bounds__(kSortThreads) sort_kernel(const SortArgs a) {
    extern __shared__ uint32_t sm[];
    let_next_start();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t *hist = sm + warp * kMaxBins;         // this warp's count of each digit
    uint32_t *total = sm + kSortWarps * kMaxBins;  // this CTA's
    uint32_t *base = total + kMaxBins;             // where this CTA's items of a digit start
    uint32_t *part = base + kMaxBins;
    const int bins = 1 << a.bits;
    // contiguous items per CTA and, inside it, per warp: order is kept
    const int64_t per_cta = (a.T + kSortCluster - 1) / kSortCluster;
    const int64_t c0 = min(a.T, per_cta * rank), c1 = min(a.T, c0 + per_cta);
    const int64_t per_warp = (c1 - c0 + kSortWarps - 1) / kSortWarps;
    const int64_t w0 = min(c1, c0 + per_warp * warp), w1 = min(c1, w0 + per_warp);
    if (rank == 0 && tid == 0) *a.n_crossing = 0;

    if (a.T <= kRanked) {
        // few enough to count, for each, the items before it: 8 threads per item
        for (int64_t i = tid; i < a.T; i += kSortThreads) {
            const int32_t id = a.ids[i];
            const bool ok = id >= 0 && id < a.V;
            sm[i] = ok ? static_cast<uint32_t>(id) : static_cast<uint32_t>(a.V);
            if (!ok && rank == 0) record_status(a.status, OOP_ERR_BAD_ID);
        }
        __syncthreads();
        const int T = static_cast<int>(a.T), i = static_cast<int>(c0) + tid / 8;
        const bool in = i < static_cast<int>(c1);
        const uint32_t key = in ? sm[i] : 0;
        uint32_t before = 0;
        for (int j = tid % 8; j < T && in; j += 8) before += sm[j] < key || (sm[j] == key && j < i);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
        if (in && tid % 8 == 0) __stcg(a.buf[0] + before, make_uint2(key, static_cast<uint32_t>(i)));
        cluster.sync();
    }
    for (int pass = 0; pass < a.passes && a.T > kRanked; ++pass) {
        // the last pass writes buf[0]
        const bool to_first = ((a.passes - pass) & 1) != 0;
        uint2 *out = to_first ? a.buf[0] : a.buf[1];
        const uint2 *in = to_first ? a.buf[1] : a.buf[0];
        const int shift = pass * a.bits;
        auto item = [&](int64_t i) -> uint2 {
            if (pass > 0) return __ldcg(in + i);
            const int32_t id = a.ids[i];
            const bool ok = id >= 0 && id < a.V;
            return make_uint2(ok ? static_cast<uint32_t>(id) : static_cast<uint32_t>(a.V),
                              static_cast<uint32_t>(i));
        };
        for (int d = lane; d < bins; d += 32) hist[d] = 0;
        __syncwarp();
        for (int64_t i = w0 + lane; i < w1; i += 32) {
            const uint2 v = item(i);
            if (pass == 0 && v.x == static_cast<uint32_t>(a.V)) record_status(a.status, OOP_ERR_BAD_ID);
            atomicAdd(hist + ((v.x >> shift) & (bins - 1)), 1u);
        }
        __syncthreads();
        if (tid < bins) {                          // counts -> starts, warp after warp
            uint32_t run = 0;
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = sm[w * kMaxBins + tid];
                sm[w * kMaxBins + tid] = run;
                run += c;
            }
            total[tid] = run;
        }
        cluster.sync();
        uint32_t before = 0, all = 0;
        if (tid < bins) {
#pragma unroll
            for (int q = 0; q < kSortCluster; ++q) {
                const uint32_t c = cluster.map_shared_rank(total, q)[tid];
                before += q < rank ? c : 0;
                all += c;
            }
        }
        uint32_t scan = all;                       // inclusive, over the digits
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += up;
        }
        if (lane == 31) part[warp] = scan;
        __syncthreads();
        const uint32_t lower = warp_sum(lane < warp ? part[lane] : 0u);
        if (tid < bins) base[tid] = lower + scan - all + before;
        __syncthreads();
        for (int64_t i0 = w0; i0 < w1; i0 += 32) {
            const int64_t i = i0 + lane;
            const uint32_t active = __ballot_sync(0xffffffffu, i < w1);
            if (i < w1) {
                const uint2 v = item(i);
                const uint32_t d = (v.x >> shift) & (bins - 1);
                const uint32_t peers = __match_any_sync(active, d);
                const uint32_t lower_lanes = peers & ((1u << lane) - 1);
                const uint32_t pos = base[d] + hist[d] + __popc(lower_lanes);
                __syncwarp(active);
                if (lower_lanes == 0) hist[d] += __popc(peers);
                __syncwarp(active);
                __stcg(out + pos, v);
            }
            __syncwarp();
        }
        cluster.sync();                            // the next pass reads what all wrote
    }
    // boundaries between chunks that a run crosses for the first time
    const uint2 *list = a.buf[0];
    const int64_t chunks = (a.T + kChunk - 1) / kChunk;
    for (int64_t c = static_cast<int64_t>(rank) * kSortThreads + tid; c + 1 < chunks;
         c += kSortCluster * kSortThreads) {
        const int64_t p0 = c * kChunk, p1 = p0 + kChunk;
        const uint32_t key = __ldcg(list + p1 - 1).x;
        if (key == static_cast<uint32_t>(a.V) || __ldcg(list + p1).x != key) continue;
        if (p0 > 0 && __ldcg(list + p0).x == key && __ldcg(list + p0 - 1).x == key) continue;
        // the last chunk that begins with key: doubling steps, then halving ones
        // (most runs cross one boundary, and every load is a round trip)
        int64_t last = c + 1, reach = 1;
        while (last + reach < chunks && __ldcg(list + (last + reach) * kChunk).x == key) {
            last += reach;
            reach *= 2;
        }
        for (; reach > 0; reach /= 2)
            if (last + reach < chunks && __ldcg(list + (last + reach) * kChunk).x == key) last += reach;
        a.crossing[atomicAdd(a.n_crossing, 1)] =
            make_uint2(static_cast<uint32_t>(c), static_cast<uint32_t>(last));
    }
}

constexpr int kSumThreads = 128;

struct SumArgs {
    const void *dy;
    int64_t nb_dy;
    const uint2 *items;                            // sorted (key, t)
    float *dw, *head, *tail;                       // parts: {M, chunks} each
    const uint2 *crossing;
    const int *n_crossing;
    int64_t M, V, T;
    float scale;
    int accumulate;
};

template <int E>
__device__ __forceinline__ void put_row(float *p, const float (&acc)[E], float scale, int accumulate) {
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = scale * acc[e];
    if (accumulate) {
        constexpr int H = E < 4 ? E : 4;
#pragma unroll
        for (int i = 0; i < E; i += H) {
            float old[H];
            load_stream<OOP_TYPE_F32, H>(p + i).get(old);
#pragma unroll
            for (int j = 0; j < H; ++j) v[i + j] += old[j];
        }
    }
    store_stream<OOP_TYPE_F32, E>(p, v);
}

template <int TYPE, int E>
__global__ void __launch_bounds__(kSumThreads) sum_rows_kernel(const SumArgs a) {
    __shared__ uint2 it[kChunk];
    wait_previous();
    let_next_start();
    const int64_t c = blockIdx.x, p0 = c * kChunk;
    const int n = static_cast<int>(min(static_cast<int64_t>(kChunk), a.T - p0));
    if (threadIdx.x < n) it[threadIdx.x] = a.items[p0 + threadIdx.x];
    const uint32_t none = static_cast<uint32_t>(a.V);      // ends of the list, ids outside
    const uint32_t prev = p0 > 0 ? a.items[p0 - 1].x : none;
    const uint32_t next = p0 + n < a.T ? a.items[p0 + n].x : none;
    __syncthreads();
    const int64_t m = (static_cast<int64_t>(blockIdx.y) * kSumThreads + threadIdx.x) * E;
    if (m >= a.M) return;
    constexpr int kBatch = 8;                      // rows in flight
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    bool from_before = it[0].x == prev;            // the run began in an earlier chunk
    for (int i0 = 0; i0 < n; i0 += kBatch) {
        Packed<TYPE, E> raw[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (i0 + j < n && it[i0 + j].x != none)
                raw[j] = load_stream<TYPE, E>(row_of<TYPE>(a.dy, a.nb_dy, it[i0 + j].y) + m);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j;
            if (i >= n || it[i].x == none) break;  // ids outside are sorted last
            float v[E];
            raw[j].get(v);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += v[e];
            const uint32_t key = it[i].x, after = i + 1 < n ? it[i + 1].x : next;
            if (i + 1 == n || after != key) {      // the run ends, or the chunk does
                const bool goes_on = after == key;
                if (from_before || goes_on)
                    store_stream<OOP_TYPE_F32, E>((from_before ? a.head : a.tail) + c * a.M + m, acc);
                else
                    put_row<E>(a.dw + static_cast<int64_t>(key) * a.M + m, acc, a.scale, a.accumulate);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = 0.f;
                from_before = false;
            }
        }
    }
}

// A CTA takes 256 columns of every gridDim.x-th run that crosses chunks; its four
// groups of 64 threads take a quarter of the run's parts each, N pieces of E
// columns per thread.
constexpr int kJoinLanes = 64, kJoinGroups = 4, kJoinCols = 256;

template <int E>
__global__ void __launch_bounds__(kJoinLanes *kJoinGroups) join_rows_kernel(const SumArgs a) {
    constexpr int N = kJoinCols / (kJoinLanes * E);
    __shared__ float part[kJoinGroups][kJoinCols];
    wait_previous();
    const int lane = threadIdx.x % kJoinLanes, group = threadIdx.x / kJoinLanes;
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kJoinCols + lane * E;
    const int n = *a.n_crossing;
    for (int r = blockIdx.x; r < n; r += gridDim.x) {
        const int64_t first = a.crossing[r].x, last = a.crossing[r].y;
        const uint32_t key = a.items[first * kChunk + kChunk - 1].x;
        const int64_t parts = last - first + 1;    // tail[first], head[first + 1 .. last]
        const int64_t k0 = first + parts * group / kJoinGroups;
        const int64_t k1 = first + parts * (group + 1) / kJoinGroups;
        float acc[N][E];
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[i][e] = 0.f;
        constexpr int kBatch = 4;                  // parts in flight
        for (int64_t k = k0; k < k1; k += kBatch) {
            Packed<OOP_TYPE_F32, E> raw[kBatch][N];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int64_t m = m0 + i * (kJoinLanes * E);
                    raw[j][i].raw = {};
                    if (k + j < k1 && m < a.M)
                        raw[j][i] = load_packed<OOP_TYPE_F32, E>((k + j == first ? a.tail : a.head) + (k + j) * a.M + m);
                }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (k + j >= k1) break;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float v[E];
                    raw[j][i].get(v);
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[i][e] += v[e];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) part[group][(i * kJoinLanes + lane) * E + e] = acc[i][e];
        __syncthreads();
        // a quarter of the columns for every group
        const int at = threadIdx.x;                // (kJoinCols threads)
        float sum = part[0][at];
#pragma unroll
        for (int g = 1; g < kJoinGroups; ++g) sum += part[g][at];
        const int64_t m = static_cast<int64_t>(blockIdx.y) * kJoinCols + at;
        const float one[1] = {sum};
        if (m < a.M) put_row<1>(a.dw + static_cast<int64_t>(key) * a.M + m, one, a.scale, a.accumulate);
        __syncthreads();
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct BackWorkspace {
    size_t buf[2], crossing, count, head, tail, bytes;
};

BackWorkspace back_workspace(int64_t M, int64_t T) {
    auto pad = [](int64_t n) { return static_cast<size_t>(n + 255) / 256 * 256; };
    const int64_t chunks = ceil_div(T, kChunk);
    BackWorkspace w;
    w.buf[0] = 0;
    w.buf[1] = w.buf[0] + pad(T * 8);
    w.crossing = w.buf[1] + pad(T * 8);
    w.count = w.crossing + pad(chunks * 8);
    w.head = w.count + 256;
    w.tail = w.head + pad(chunks * M * 4);
    w.bytes = w.tail + pad(chunks * M * 4);
    return w;
}

template <int TYPE, int E>
cudaError_t launch_sums(const SumArgs &a, cudaStream_t st) {
    const int64_t chunks = ceil_div(a.T, kChunk);
    const int64_t tiles = ceil_div(a.M, kSumThreads * E);
    const cudaError_t e = launch_dependent(
        sum_rows_kernel<TYPE, E>, dim3(static_cast<unsigned>(chunks), static_cast<unsigned>(tiles)),
        kSumThreads, 0, st, a);
    if (e != cudaSuccess || chunks < 2) return e;
    constexpr int J = E > 4 ? 4 : E;
    return launch_dependent(join_rows_kernel<J>,
                            dim3(static_cast<unsigned>(std::min<int64_t>(chunks - 1, 256)),
                                 static_cast<unsigned>(ceil_div(a.M, kJoinCols))),
                            kJoinLanes * kJoinGroups, 0, st, a);
}

using RowsKernel = void (*)(const void *, int64_t, const int32_t *, void *, int64_t, int64_t,
                            int64_t, int64_t, float, int *);

// Below this, a CTA takes one token (as many CTAs as there are, for latency).
constexpr int64_t kManyTokens = 2048;

struct RowsChoice {
    RowsKernel kernel;
    int E, R;
};

template <int TYPE, int OUT>
RowsChoice rows_kernel(bool wide, bool many) {
    // a vector is 16 bytes of the narrower type; quantised rows are decoded
    // four elements at a time
    constexpr int E = TYPE == OOP_TYPE_F32 || OUT == OOP_TYPE_F32 || !is_plain_type<TYPE>() ? 4 : 8;
    if constexpr (is_plain_type<TYPE>()) {
        if (many && wide) return {get_rows_kernel<TYPE, OUT, E, 4>, E, 4};
        if (many) return {get_rows_kernel<TYPE, OUT, 1, 4>, 1, 4};
    }
    if (wide) return {get_rows_kernel<TYPE, OUT, E, 1>, E, 1};
    return {get_rows_kernel<TYPE, OUT, 1, 1>, 1, 1};
}

template <int TYPE>
RowsChoice rows_kernel(int out, bool wide, bool many) {
    switch (out) {
    case OOP_TYPE_F32: return rows_kernel<TYPE, OOP_TYPE_F32>(wide, many);
    case OOP_TYPE_F16: return rows_kernel<TYPE, OOP_TYPE_F16>(wide, many);
    default: return rows_kernel<TYPE, OOP_TYPE_BF16>(wide, many);
    }
}

RowsChoice rows_kernel(int type, int out, bool wide, bool many) {
    switch (type) {
#define OOP_ROWS_CASE(T) \
    case T: return rows_kernel<T>(out, wide, many);
    OOP_ROWS_CASE(OOP_TYPE_F32)
    OOP_ROWS_CASE(OOP_TYPE_F16)
    OOP_ROWS_CASE(OOP_TYPE_BF16)
    OOP_ROWS_CASE(OOP_TYPE_Q4_0)
    OOP_ROWS_CASE(OOP_TYPE_Q4_1)
    OOP_ROWS_CASE(OOP_TYPE_Q5_0)
    OOP_ROWS_CASE(OOP_TYPE_Q5_1)
    OOP_ROWS_CASE(OOP_TYPE_Q8_0)
    OOP_ROWS_CASE(OOP_TYPE_Q2_K)
    OOP_ROWS_CASE(OOP_TYPE_Q3_K)
    OOP_ROWS_CASE(OOP_TYPE_Q4_K)
    OOP_ROWS_CASE(OOP_TYPE_Q5_K)
    OOP_ROWS_CASE(OOP_TYPE_Q6_K)
#undef OOP_ROWS_CASE
    default: return {nullptr, 1, 1};
    }
}

int check_rows(const int64_t ne[2], int64_t n_ids) {
    if (!ne) return OOP_ERR_NULL;
    const int rc = check_extent(ne[0], ne[1]);
    if (rc != OOP_OK) return rc;
    if (n_ids < 0 || n_ids > 0x7fffffffLL || ne[1] > 0x7fffffffLL) return OOP_ERR_SHAPE;
    if (ne[0] > (1 << 20)) return OOP_ERR_SHAPE;             // column tiles ride grid.y
    return check_extent(ne[0], n_ids);
}

}  // namespace
}  // namespace oop

using namespace oop;

extern "C" {

int oop_get_rows(const void *table, int table_type, int64_t nb_table, const int32_t *ids,
                 void *dst, int dst_type, int64_t nb_dst, const int64_t ne_table[2],
                 int64_t n_ids, float scale, void *stream) {
    g_kernel_launches = 0;
    int rc = check_rows(ne_table, n_ids);
    if (rc != OOP_OK) return rc;
    const int qk = type_block_elems(table_type);
    if (qk < 0 || !plain_size(dst_type)) return OOP_ERR_TYPE;
    const int64_t M = ne_table[0], V = ne_table[1];
    if (M % qk != 0) return OOP_ERR_SHAPE;
    const int size = table_type == OOP_TYPE_F32 ? 4 : 2;      // every block is of an even size
    rc = check_row_stride(M / qk * type_block_bytes(table_type), V, nb_table, size, false);
    if (rc != OOP_OK) return rc;
    rc = check_row_stride(M * plain_size(dst_type), n_ids, nb_dst, plain_size(dst_type), true);
    if (rc != OOP_OK) return rc;
    if (M == 0 || n_ids == 0) return OOP_OK;
    if ((rc = check_pointer(dst, plain_size(dst_type))) != OOP_OK) return rc;
    if ((rc = check_pointer(ids, 4)) != OOP_OK) return rc;
    if (V > 0 && (rc = check_pointer(table, size)) != OOP_OK) return rc;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    // wide accesses need 16-byte aligned rows (8 columns at most make one);
    // a quantised row is read by the block, so only dst matters
    const bool plain = qk == 1;
    const bool wide = M % 8 == 0 && is_aligned(dst, 16) && nb_dst % 16 == 0 &&
                      (!plain || (is_aligned(table, 16) && nb_table % 16 == 0));
    const bool many = n_ids >= kManyTokens;
    const RowsChoice k = rows_kernel(table_type, dst_type, wide, many);
    const int64_t tiles = ceil_div(M, static_cast<int64_t>(kThreads) * k.E);
    k.kernel<<<dim3(static_cast<unsigned>(ceil_div(n_ids, k.R)), static_cast<unsigned>(tiles)),
               kThreads, 0, static_cast<cudaStream_t>(stream)>>>(table, nb_table, ids, dst, nb_dst,
                                                                 M, V, n_ids, scale, status);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) g_kernel_launches = 1;
    return cuda_status(e);
}

size_t oop_get_rows_back_workspace_size(const int64_t ne_table[2], int64_t n_ids) {
    if (check_rows(ne_table, n_ids) != OOP_OK) return 0;
    if (ne_table[0] == 0 || ne_table[1] == 0 || n_ids == 0) return 0;
    return back_workspace(ne_table[0], n_ids).bytes;
}

int oop_get_rows_back(const void *dy, int dy_type, int64_t nb_dy, const int32_t *ids,
                      float *dtable, const int64_t ne_table[2], int64_t n_ids, float scale,
                      int accumulate, void *workspace, size_t workspace_bytes, void *stream) {
    g_kernel_launches = 0;
    int rc = check_rows(ne_table, n_ids);
    if (rc != OOP_OK) return rc;
    if (!gradient_type(dy_type)) return OOP_ERR_TYPE;
    const int64_t M = ne_table[0], V = ne_table[1];
    const int size = plain_size(dy_type);
    rc = check_row_stride(M * size, n_ids, nb_dy, size, false);
    if (rc != OOP_OK) return rc;
    if (M == 0 || V == 0) return OOP_OK;
    if ((rc = check_pointer(dtable, 4)) != OOP_OK) return rc;
    if (n_ids > 0) {
        if ((rc = check_pointer(dy, size)) != OOP_OK) return rc;
        if ((rc = check_pointer(ids, 4)) != OOP_OK) return rc;
    }
    const size_t need = oop_get_rows_back_workspace_size(ne_table, n_ids);
    if (need > 0 && (!workspace || workspace_bytes < need || !is_aligned(workspace, 256)))
        return OOP_ERR_WORKSPACE;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (n_ids == 0)                                          // empty sums
        return accumulate ? OOP_OK
                          : cuda_status(cudaMemsetAsync(dtable, 0, static_cast<size_t>(M * V) * 4, st));
    // 16 bytes of dy are 4 or 8 columns; dtable's rows follow dtable
    const bool wide = M % (16 / size) == 0 && is_aligned(dy, 16) && nb_dy % 16 == 0 &&
                      is_aligned(dtable, 16);
    char *ws = static_cast<char *>(workspace);
    const BackWorkspace w = back_workspace(M, n_ids);
    const SortPlan plan = sort_plan(V);
    SortArgs sa = {ids,
                   {reinterpret_cast<uint2 *>(ws + w.buf[0]), reinterpret_cast<uint2 *>(ws + w.buf[1])},
                   reinterpret_cast<uint2 *>(ws + w.crossing), reinterpret_cast<int *>(ws + w.count),
                   n_ids, V, plan.bits, plan.passes, status};
    cudaError_t e = allow_smem<sort_kernel>();
    if (e != cudaSuccess) return cuda_status(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSortCluster);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = kSortSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSortCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, sort_kernel, sa);
    if (e == cudaSuccess && !accumulate)
        e = launch_dependent(fill_zero_kernel,
                             dim3(static_cast<unsigned>(ceil_div(M * V, 8 * kThreads))), kThreads, 0,
                             st, dtable, M * V);
    if (e != cudaSuccess) return cuda_status(e);
    const SumArgs su = {dy, nb_dy, sa.buf[0], dtable, reinterpret_cast<float *>(ws + w.head),
                        reinterpret_cast<float *>(ws + w.tail), sa.crossing, sa.n_crossing, M, V,
                        n_ids, scale, accumulate};
    if (dy_type == OOP_TYPE_F32)
        e = wide ? launch_sums<OOP_TYPE_F32, 4>(su, st) : launch_sums<OOP_TYPE_F32, 1>(su, st);
    else
        e = wide ? launch_sums<OOP_TYPE_BF16, 8>(su, st) : launch_sums<OOP_TYPE_BF16, 1>(su, st);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) g_kernel_launches = 2 + !accumulate + (n_ids > kChunk);
    return cuda_status(e);
}

}  // extern "C"
