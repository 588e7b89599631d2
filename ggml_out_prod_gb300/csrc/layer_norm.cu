// layer_norm.cu -- layer norm over the rows of {M, T}, forward and backward.
// Both passes are bound by memory: forward each element is read and written
// once, backward x and dy are read once and dx written once, and dw and db come
// out of the same pass.
//
//   y  = (x - mean) * rstd * w + b,   rstd = (var + eps)^(-1/2)
//   g  = dy * w,  xh = (x - mean) * rstd
//   dx = rstd * (g - mean(g) - xh * mean(g * xh))
//   dw = sum over rows of dy * xh,   db = sum over rows of dy
//
// var is the mean of (x - mean)^2, taken after the mean is known: the
// difference of the mean square and the squared mean cancels for rows far from
// zero.
#include <algorithm>
#include <cmath>

#include "oop_internal.cuh"
#include "rows.cuh"
#include "tc_ptx.cuh"

namespace oop {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kSlices = 152;     // CTAs of the row kernels, one per SM: slices of dw and db
static_assert(kSlices % (kThreads / 32) == 0);
constexpr int kMaxThreads = 512;     // of a row kernel's CTA: 128 registers each
constexpr int kSmem = 220 * 1024;    // of a CTA that has an SM to itself

struct NormArgs {
    const void *x, *w, *b;
    void *y;
    float *mean, *rstd;
    int64_t nb_x, nb_y, M, T;
    int w_type;
    int width, pieces, groups;       // threads per row, pieces of a thread, rows at once
    float eps;
};

// Column m0 .. m0 + E - 1 of a parameter of a run-time type (E = 1, or a 32-byte
// aligned parameter and m0 % E == 0).
template <int E>
__device__ __forceinline__ void load_params(const void *p, int type, int64_t m0, float (&v)[E]) {
    if (type == OOP_TYPE_F32 && E == 8) {
        // one 32-byte access: as two of 16 bytes, a warp's lanes would lie 32
        // bytes apart in each and take twice the cache's bandwidth
        const float *q = static_cast<const float *>(p) + m0;
        asm("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=f"(v[0]), "=f"(v[1 % E]), "=f"(v[2 % E]), "=f"(v[3 % E]), "=f"(v[4 % E]), "=f"(v[5 % E]),
              "=f"(v[6 % E]), "=f"(v[7 % E])
            : "l"(q));
    } else if (type == OOP_TYPE_F32) {
        constexpr int H = E < 4 ? E : 4;
#pragma unroll
        for (int i = 0; i < E; i += H) {
            float part[H];
            load_packed<OOP_TYPE_F32, H>(static_cast<const float *>(p) + m0 + i).get(part);
#pragma unroll
            for (int j = 0; j < H; ++j) v[i + j] = part[j];
        }
    } else if (type == OOP_TYPE_F16) {
        load_packed<OOP_TYPE_F16, E>(static_cast<const __half *>(p) + m0).get(v);
    } else {
        load_packed<OOP_TYPE_BF16, E>(static_cast<const __nv_bfloat16 *>(p) + m0).get(v);
    }
}

// A thread's own piece of shared memory, filled behind its back: copies of 4,
// 8 or 16 bytes, committed row by row.
template <int BYTES>
__device__ __forceinline__ void copy_async(void *smem, const void *p) {
    const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(p) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s), "l"(p), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `left` (0 .. 3) committed rows are still on their way.
__device__ __forceinline__ void wait_copies(int left) {
    if (left == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (left == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (left == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// Columns of one thread in the backward pass: a row's two reductions and its
// bookkeeping cost a warp as much as 20 columns do.
constexpr int kCols = 32;
constexpr int kMaxStages = 4;

// A row's threads: `width` of them, whole warps, in a CTA that has several rows in
// work, a group of threads each.
struct Place {
    int M, threads, width, group, lane, warps, warp0;
    int full, rest;                  // singles: every lane has `full` of them, `rest` lanes one more

    __device__ __forceinline__ Place(int64_t M_, int width_)
        : M(static_cast<int>(M_)), threads(blockDim.x), width(width_), group(threadIdx.x / width_),
          lane(threadIdx.x - group * width_), warps(width_ >> 5), warp0(group * (width_ >> 5)),
          full(M / width_), rest(M - full * width_) {}
    // the thread's i-th piece of E columns starts here
    template <int E>
    __device__ __forceinline__ int column(int i) const { return (i * width + lane) * E; }
    // whether it lies in the row
    template <int E>
    __device__ __forceinline__ bool has(int i) const {
        return E == 1 ? i < full || (i == full && lane < rest) : column<E>(i) < M;
    }
};

// A thread's columns come in units that are there or not as a whole: a
// vector of E, or two singles (of which the second may be missing).
template <int E>
struct Units {
    static constexpr int kSize = E == 1 ? 2 : E, kPairs = kSize / 2;
    static constexpr int kPieces = kSize / E;        // pieces per unit
};

// Where a matrix lies: rows are copied by the 16 bytes, and those at a row's ends
// may hold a neighbour's elements, but nothing before the first row or behind
// the last one is touched.
struct Extent {
    const char *begin, *end;
    __device__ __forceinline__ Extent(const void *p, int64_t nb, int64_t T, int64_t row_bytes)
        : begin(static_cast<const char *>(p)), end(begin + (T - 1) * nb + row_bytes) {}
};

// Bytes of a row of singles in shared memory: the 16-byte pieces it may touch.
__host__ __device__ constexpr int row_room(int64_t M, int size) {
    return static_cast<int>((M * size + 15 + 15) / 16 * 16);
}

// Copies a row as it lies, from the 16-byte boundary at or below its start, by
// `width` threads; element m is then at (row & 15) + m * size.
template <int TYPE>
__device__ __forceinline__ void copy_row(char *to, const char *row, int64_t row_bytes, const Extent &all, int lane,
                                         int width) {
    using S = typename Plain<TYPE>::S;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
    const char *from = row - off;
    const int n = static_cast<int>((off + row_bytes + 15) / 16);
    for (int c = lane; c < n; c += width) {
        const char *p = from + c * 16;
        if (p >= all.begin && p + 16 <= all.end) {
            copy_async<16>(to + c * 16, p);
        } else {                                     // the matrix's first or last elements
            for (int k = 0; k < 16; k += sizeof(S))
                if (p + k >= row && p + k < row + row_bytes)
                    *reinterpret_cast<S *>(to + c * 16 + k) = *reinterpret_cast<const S *>(p + k);
        }
    }
}

// One operand's rows, staged as {stages, columns / E, threads} pieces, each read
// by the thread that copied it; or (E = 1) as {stages} whole rows of one group,
// read by all its threads.
template <int TYPE, int E>
struct Staged {
    static constexpr int kBytes = E * plain_size(TYPE);
    char *mine;                                      // this thread's piece 0 of stage 0
    int stage_bytes, piece_bytes;

    __device__ __forceinline__ Staged(char *base, const Place &p, const void *, int64_t, int64_t, int)
        : mine(base + threadIdx.x * kBytes), stage_bytes(p.threads * kCols * plain_size(TYPE)),
          piece_bytes(p.threads * kBytes) {}
    // bytes of all stages
    __device__ __forceinline__ int room(const Place &, int stages) const { return stages * stage_bytes; }
    __device__ __forceinline__ void issue(const char *row, int st, const Place &p) const {
        char *to = mine + st * stage_bytes;
        row += p.lane * kBytes;
#pragma unroll
        for (int i = 0; i < kCols / E; ++i)
            if (p.column<E>(i) < p.M) copy_async<kBytes>(to + i * piece_bytes, row + i * (p.width * kBytes));
    }
    // Unit u as pairs.
    __device__ __forceinline__ void get(int u, int st, const char *, const Place &, uint64_t (&v)[E / 2]) const {
        Packed<TYPE, E> r;
        r.raw = *reinterpret_cast<const decltype(r.raw) *>(mine + st * stage_bytes + u * piece_bytes);
        float f[E];
        r.get(f);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) v[j] = ptx::pack2(f[2 * j], f[2 * j + 1]);
    }
};

template <int TYPE>
struct Staged<TYPE, 1> {
    static constexpr int kBytes = plain_size(TYPE);
    char *rows;                                      // this group's
    int stage_bytes, row_bytes;
    Extent all;

    __device__ __forceinline__ Staged(char *base, const Place &p, const void *x, int64_t nb, int64_t T, int stages)
        : rows(base + p.group * stages * row_room(p.M, kBytes)), stage_bytes(row_room(p.M, kBytes)),
          row_bytes(p.M * kBytes), all(x, nb, T, row_bytes) {}
    __device__ __forceinline__ int room(const Place &p, int stages) const {
        return (p.threads / p.width) * stages * stage_bytes;
    }
    __device__ __forceinline__ void issue(const char *row, int st, const Place &p) const {
        copy_row<TYPE>(rows + st * stage_bytes, row, row_bytes, all, p.lane, p.width);
    }
    // Unit u as a pair; a missing second single is 0.
    __device__ __forceinline__ void get(int u, int st, const char *row, const Place &p, uint64_t (&v)[1]) const {
        const auto *q = reinterpret_cast<const typename Plain<TYPE>::S *>(
            rows + st * stage_bytes + (reinterpret_cast<uintptr_t>(row) & 15));
        const int m = p.column<1>(2 * u), n = p.column<1>(2 * u + 1);
        v[0] = ptx::pack2(to_float(q[m]), p.has<1>(2 * u + 1) ? to_float(q[n]) : 0.f);
    }
};

// Whether unit u's first column is inside the row (and so all of it, but for a
// second single).
template <int E>
__device__ __forceinline__ bool has_unit(int u, const Place &p) {
    return p.has<E>(u * Units<E>::kPieces);
}

// Unit u of a row of results (row: the address of the thread's first piece).
template <int TYPE, int E>
__device__ __forceinline__ void put_unit(char *row, int u, const Place &p, const uint64_t (&v)[Units<E>::kPairs]) {
    auto *out = reinterpret_cast<typename Plain<TYPE>::S *>(row);
    float f[Units<E>::kSize];
#pragma unroll
    for (int j = 0; j < Units<E>::kPairs; ++j) ptx::unpack2(v[j], f[2 * j], f[2 * j + 1]);
#pragma unroll
    for (int k = 0; k < Units<E>::kPieces; ++k) {
        const int i = u * Units<E>::kPieces + k;
        float part[E];
#pragma unroll
        for (int e = 0; e < E; ++e) part[e] = f[k * E + e];
        if (k == 0 || p.has<E>(i)) store_stream<TYPE, E>(out + i * (p.width * E), part);
    }
}

__device__ __forceinline__ uint64_t both(float v) { return ptx::pack2(v, v); }
__device__ __forceinline__ float add_halves(uint64_t v) {
    float lo, hi;
    ptx::unpack2(v, lo, hi);
    return lo + hi;
}

// One value of each of a row's warps in every lane w < warps of all of them.
__device__ __forceinline__ float2 exchange(float2 v, const Place &p, float2 *red, int &odd) {
    float2 *now = red + odd * 32;                    // the other half may still be read
    if ((threadIdx.x & 31) == 0) now[threadIdx.x >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(p.group + 1), "r"(p.width) : "memory");
    odd ^= 1;
    const int lane = threadIdx.x & 31;
    return lane < p.warps ? now[p.warp0 + lane] : make_float2(0.f, 0.f);
}

// 2 * N floats, 16-byte aligned.
template <int N>
__device__ __forceinline__ void put_floats(float *out, const uint64_t (&v)[N]) {
#pragma unroll
    for (int j = 0; j + 1 < N; j += 2) {
        float4 q;
        ptx::unpack2(v[j], q.x, q.y);
        ptx::unpack2(v[j + 1], q.z, q.w);
        *reinterpret_cast<float4 *>(out + 2 * j) = q;
    }
}

// w or b (`none` where NULL) to shared memory as floats, by the whole CTA: in the
// order in which a row's threads read it, 16 bytes per lane in turn, so that no two
// lanes of an access meet in a bank.  The loads go out four at a time, since the
// first row waits for them.
template <int E>
__device__ __forceinline__ void stage_params(float *to, const void *q, int type, float none, int M, int width) {
    constexpr int kAhead = 4;
    const int units = M / E, threads = blockDim.x;
    for (int c0 = threadIdx.x; c0 < units; c0 += kAhead * threads) {
        float v[kAhead][E];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
#pragma unroll
            for (int e = 0; e < E; ++e) v[k][e] = none;
            if (q && c0 + k * threads < units) load_params<E>(q, type, int64_t(c0 + k * threads) * E, v[k]);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int c = c0 + k * threads;
            if (c >= units) break;
            if constexpr (E == 1) {
                to[c] = v[k][0];
            } else {
                const int i = c / width, lane = c - i * width;
#pragma unroll
                for (int h = 0; h < E / 4; ++h)
                    *reinterpret_cast<float4 *>(to + ((i * (E / 4) + h) * width + lane) * 4) =
                        make_float4(v[k][4 * h], v[k][4 * h + 1], v[k][4 * h + 2], v[k][4 * h + 3]);
            }
        }
    }
}

// A row held in registers by `width` threads, n pieces of E columns each (of at
// most NV).  FULL: every lane has n whole pieces.
template <int XT, int E, int NV, bool FULL>
struct HeldRow {
    Packed<XT, E> raw[NV];
    bool last;                       // the lane has the last of the n pieces too

    __device__ __forceinline__ HeldRow(int n, const Place &p) : last(p.column<E>(n - 1) < p.M) {}
    __device__ __forceinline__ bool has(int i, int n) const { return FULL || i + 1 < n || last; }
    // f(i, values) for each of the thread's pieces.
    template <class F>
    __device__ __forceinline__ void each(int n, F f) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (i >= n) break;
            float v[E];
            raw[i].get(v);
            if (has(i, n)) f(i, v);
        }
    }
    __device__ __forceinline__ float sum(int n) const {
        if constexpr (E == 1) {
            float s = 0.f;
            each(n, [&](int, const float (&v)[E]) { s += v[0]; });
            return warp_sum(s);
        } else {
            uint64_t acc[2] = {0, 0};
            each(n, [&](int, const float (&v)[E]) {
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    acc[(e / 2) & 1] = ptx::add2(acc[(e / 2) & 1], ptx::pack2(v[e], v[e + 1]));
            });
            return warp_sum(add_halves(ptx::add2(acc[0], acc[1])));
        }
    }
    __device__ __forceinline__ float squares(int n, float mean) const {
        if constexpr (E == 1) {
            float s = 0.f;
            each(n, [&](int, const float (&v)[E]) { s = fmaf(v[0] - mean, v[0] - mean, s); });
            return warp_sum(s);
        } else {
            uint64_t acc[2] = {0, 0};
            const uint64_t m2 = both(mean);
            each(n, [&](int, const float (&v)[E]) {
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const uint64_t d = ptx::sub2(ptx::pack2(v[e], v[e + 1]), m2);
                    acc[(e / 2) & 1] = ptx::fma2(d, d, acc[(e / 2) & 1]);
                }
            });
            return warp_sum(add_halves(ptx::add2(acc[0], acc[1])));
        }
    }
};

// Columns of warp k of a row.
template <int E, bool FULL>
__device__ __forceinline__ float warp_columns(int k, int n, const Place &p) {
    if (FULL) return static_cast<float>(n * 32 * E);
    int c = 0;
    for (int i = 0; i < n; ++i) c += max(0, min(32 * E, p.M - (i * p.width + k * 32) * E));
    return static_cast<float>(c);
}

// (mean, rstd) of a row.  Rows that several warps share exchange once: each warp
// takes its own mean and the squares about it, and the row's are those of the
// warps' means and theirs, so nothing cancels whatever the mean (a sum of
// squares would).  `meet` is the barrier of the row's warps.
template <int XT, int E, int NV, bool FULL, class Meet>
__device__ __forceinline__ float2 moments(const HeldRow<XT, E, NV, FULL> &row, int n, const Place &p, float eps,
                                          float own, float theirs, float2 *red, Meet meet) {
    const float s = row.sum(n);
    float mean = own > 0.f ? s / own : 0.f;
    float sq = row.squares(n, mean);
    if (p.warps > 1) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) red[threadIdx.x >> 5] = make_float2(s, sq);
        meet();
        const float2 r = lane < p.warps ? red[p.warp0 + lane] : make_float2(0.f, 0.f);
        mean = warp_sum(r.x) / static_cast<float>(p.M);
        const float d = theirs > 0.f ? r.x / theirs - mean : 0.f;
        sq = warp_sum(fmaf(theirs * d, d, r.y));
    }
    return make_float2(mean, rsqrtf(sq / static_cast<float>(p.M) + eps));
}

// The forward pass of few rows, and of rows that come in singles: a row per
// `width` threads, every load before the first use.
template <int XT, int YT, int E, int NV, bool FULL>
__global__ void __launch_bounds__(NV > 16 ? 512 : 1024) norm_kernel(const NormArgs a) {
    __shared__ float2 red[32];
    const Place p(a.M, a.width);
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / a.width) + p.group;
    const bool in = t < a.T;
    if (!in && p.warps == 1) return;
    const auto *x = row_of<XT>(a.x, a.nb_x, in ? t : 0) + p.lane * E;
    const int step = p.width * E, n = a.pieces, lane = threadIdx.x & 31;
    HeldRow<XT, E, NV, FULL> row(n, p);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (i >= n) break;
        if (row.has(i, n)) row.raw[i] = load_stream<XT, E>(x + i * step);
    }
    const float own = warp_columns<E, FULL>(p.lane >> 5, n, p);
    const float theirs = lane < p.warps ? warp_columns<E, FULL>(lane, n, p) : 0.f;
    const float2 mr = moments(row, n, p, a.eps, own, theirs, red, [] { __syncthreads(); });
    if (!in) return;
    auto *y = row_of<YT>(a.y, a.nb_y, t) + p.lane * E;
    // parameters a few pieces ahead of their use: singly, each would be a wait
    constexpr int kAhead = E == 1 ? (NV < 8 ? NV : 8) : 2;
#pragma unroll
    for (int i0 = 0; i0 < NV; i0 += kAhead) {
        if (i0 >= n) break;
        float w[kAhead][E], b[kAhead][E];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                w[j][e] = 1.f;
                b[j][e] = 0.f;
            }
            if (i >= n || !row.has(i, n)) continue;
            if (a.w) load_params<E>(a.w, a.w_type, p.column<E>(i), w[j]);
            if (a.b) load_params<E>(a.b, a.w_type, p.column<E>(i), b[j]);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j;
            if (i >= n || !row.has(i, n)) continue;
            float v[E];
            row.raw[i].get(v);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = fmaf((v[e] - mr.x) * mr.y, w[j][e], b[j][e]);
            store_stream<YT, E>(y + i * step, v);
        }
    }
    if (p.lane == 0) {
        if (a.mean) a.mean[t] = mr.x;
        if (a.rstd) a.rstd[t] = mr.y;
    }
}

// The forward pass of many rows (bf16, 16384 x 5120: 60 us, 5.6 TB/s, 83% of the
// measured copy rate; a CTA per four rows with w and b from L1: 76 us).  One CTA per
// SM keeps w and b in shared memory and takes row after row; a warp has as much of
// a row as its registers hold (20 vectors a lane), so that a reduction is paid for
// by up to 160 columns a lane and most rows need no barrier.  A lane copies its
// pieces of its next row to shared memory from when it has taken the current one
// into registers: there is always a row per warp on its way.  For narrow rows that
// is little (bf16, 131072 x 128: 51 us, 20% of the copy rate; f32 41 us, 48%).
template <int XT, int YT, int E, int NV, bool FULL>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_many_kernel(const NormArgs a) {
    constexpr int kBytes = E * plain_size(XT);
    extern __shared__ __align__(16) char sm[];
    const Place p(a.M, a.width);
    float2 *red = reinterpret_cast<float2 *>(sm);                    // {2, 16}
    float *ws = reinterpret_cast<float *>(sm + 256), *bs = ws + a.pieces * a.width * E;
    char *mine = reinterpret_cast<char *>(bs + a.pieces * a.width * E) + threadIdx.x * kBytes;
    const int n = a.pieces, lane = threadIdx.x & 31, piece = p.threads * kBytes;
    const int64_t step = static_cast<int64_t>(gridDim.x) * a.groups;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * a.groups + p.group;
    const char *x = static_cast<const char *>(a.x) + r0 * a.nb_x + p.lane * kBytes;
    char *y = static_cast<char *>(a.y) + r0 * a.nb_y + p.lane * (E * plain_size(YT));
    HeldRow<XT, E, NV, FULL> row(n, p);
    auto issue = [&](int64_t t) {
        if (t < a.T) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i >= n) break;
                if (row.has(i, n))
                    copy_async<kBytes>(mine + i * piece, x + i * (p.width * kBytes));
            }
        }
        commit_copies();
        x += step * a.nb_x;
    };
    issue(r0);
    stage_params<E>(ws, a.w, a.w_type, 1.f, p.M, p.width);
    stage_params<E>(bs, a.b, a.w_type, 0.f, p.M, p.width);
    __syncthreads();
    const float own = warp_columns<E, FULL>(p.lane >> 5, n, p);
    const float theirs = lane < p.warps ? warp_columns<E, FULL>(lane, n, p) : 0.f;
    int odd = 0;
    for (int64_t t = r0; t < a.T; t += step) {
        wait_copies(0);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (i >= n) break;
            row.raw[i].raw = *reinterpret_cast<const decltype(row.raw[i].raw) *>(mine + i * piece);
        }
        issue(t + step);
        const float2 mr = moments(row, n, p, a.eps, own, theirs, red + odd, [&] {
            asm volatile("bar.sync %0, %1;" ::"r"(p.group + 1), "r"(p.width) : "memory");
        });
        odd ^= 16;                                   // the other half may still be read
        const uint64_t mean = both(mr.x), rstd = both(mr.y);
        row.each(n, [&](int i, float (&v)[E]) {
#pragma unroll
            for (int h = 0; h < E / 4; ++h) {
                const int at = ((i * (E / 4) + h) * p.width + p.lane) * 4;
                const float4 w = *reinterpret_cast<const float4 *>(ws + at);
                const float4 b = *reinterpret_cast<const float4 *>(bs + at);
                uint64_t lo = ptx::pack2(v[4 * h], v[4 * h + 1]), hi = ptx::pack2(v[4 * h + 2], v[4 * h + 3]);
                lo = ptx::fma2(ptx::mul2(ptx::sub2(lo, mean), rstd), ptx::pack2(w.x, w.y), ptx::pack2(b.x, b.y));
                hi = ptx::fma2(ptx::mul2(ptx::sub2(hi, mean), rstd), ptx::pack2(w.z, w.w), ptx::pack2(b.z, b.w));
                ptx::unpack2(lo, v[4 * h], v[4 * h + 1]);
                ptx::unpack2(hi, v[4 * h + 2], v[4 * h + 3]);
            }
            store_stream<YT, E>(reinterpret_cast<typename Plain<YT>::S *>(y) + i * (p.width * E), v);
        });
        if (p.lane == 0) {
            if (a.mean) a.mean[t] = mr.x;
            if (a.rstd) a.rstd[t] = mr.y;
        }
        y += step * a.nb_y;
    }
}

// The forward pass of many rows that are not aligned.  As above, but a row is
// copied as it lies, by all of its threads together, and they read it from
// shared memory element by element, neighbouring lanes neighbouring elements:
// alignment then costs nothing but narrow reads and stores.
template <int XT, int YT>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_odd_kernel(const NormArgs a) {
    using SX = typename Plain<XT>::S;
    extern __shared__ __align__(16) char sm[];
    const Place p(a.M, a.width);
    const int room = row_room(p.M, sizeof(SX)), lane = threadIdx.x & 31;
    float2 *red = reinterpret_cast<float2 *>(sm);                    // {2, 16}
    char *rows = sm + 256 + p.group * 2 * room;
    float *ws = reinterpret_cast<float *>(sm + 256 + a.groups * 2 * room), *bs = ws + p.M;
    const unsigned step = gridDim.x * a.groups, T = static_cast<unsigned>(a.T);
    const unsigned r0 = blockIdx.x * a.groups + p.group;
    const int64_t up_x = step * a.nb_x, up_y = step * a.nb_y, row_bytes = a.M * int64_t(sizeof(SX));
    const Extent all(a.x, a.nb_x, a.T, row_bytes);
    const char *x = static_cast<const char *>(a.x) + r0 * a.nb_x;
    char *y = static_cast<char *>(a.y) + r0 * a.nb_y;
    auto meet = [&] {
        if (p.warps > 1) asm volatile("bar.sync %0, %1;" ::"r"(p.group + 1), "r"(p.width) : "memory");
        else __syncwarp();
    };
    if (r0 < T) copy_row<XT>(rows, x, row_bytes, all, p.lane, p.width);
    commit_copies();
    stage_params<1>(ws, a.w, a.w_type, 1.f, p.M, p.width);
    stage_params<1>(bs, a.b, a.w_type, 0.f, p.M, p.width);
    __syncthreads();
    // columns of this warp, and of warp `lane` of the row: every width-th 32
    auto columns = [&](int k) {
        int c = 0;
        for (int m = k * 32; m < p.M; m += p.width) c += min(32, p.M - m);
        return static_cast<float>(c);
    };
    const float own = columns(p.lane >> 5), theirs = lane < p.warps ? columns(lane) : 0.f;
    int st = 0;
    for (unsigned t = r0; t < T; t += step, st ^= 1) {
        wait_copies(0);
        meet();                                      // the row is there, the one before it done with
        const SX *v = reinterpret_cast<const SX *>(rows + st * room + (reinterpret_cast<uintptr_t>(x) & 15));
        x += up_x;
        if (t + step < T) copy_row<XT>(rows + (st ^ 1) * room, x, row_bytes, all, p.lane, p.width);
        commit_copies();
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        int m = p.lane;
        for (; m + 3 * p.width < p.M; m += 4 * p.width)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += to_float(v[m + j * p.width]);
        for (; m < p.M; m += p.width) s[0] += to_float(v[m]);
        const float sum = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
        float mean = own > 0.f ? sum / own : 0.f;
        s[0] = s[1] = s[2] = s[3] = 0.f;
        for (m = p.lane; m + 3 * p.width < p.M; m += 4 * p.width)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float d = to_float(v[m + j * p.width]) - mean;
                s[j] = fmaf(d, d, s[j]);
            }
        for (; m < p.M; m += p.width) {
            const float d = to_float(v[m]) - mean;
            s[0] = fmaf(d, d, s[0]);
        }
        float sq = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
        if (p.warps > 1) {
            float2 *now = red + st * 16;             // the other half may still be read
            if (lane == 0) now[threadIdx.x >> 5] = make_float2(sum, sq);
            meet();
            const float2 r = lane < p.warps ? now[p.warp0 + lane] : make_float2(0.f, 0.f);
            mean = warp_sum(r.x) / static_cast<float>(p.M);
            const float d = theirs > 0.f ? r.x / theirs - mean : 0.f;
            sq = warp_sum(fmaf(theirs * d, d, r.y));
        }
        const float rstd = rsqrtf(sq / static_cast<float>(p.M) + a.eps);
        auto *out = reinterpret_cast<typename Plain<YT>::S *>(y);
        for (m = p.lane; m + 3 * p.width < p.M; m += 4 * p.width)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = m + j * p.width;
                __stcs(out + k, from_float<YT>(fmaf((to_float(v[k]) - mean) * rstd, ws[k], bs[k])));
            }
        for (; m < p.M; m += p.width) __stcs(out + m, from_float<YT>(fmaf((to_float(v[m]) - mean) * rstd, ws[m], bs[m])));
        if (p.lane == 0) {
            if (a.mean) a.mean[t] = mean;
            if (a.rstd) a.rstd[t] = rstd;
        }
        y += up_y;
    }
}

// Rows of which no two fit (of the many rows that norm_many_kernel takes, not even
// one): one CTA per row, read three times, the second and third time from L2, by
// single elements.  2048 rows: f32 x 20480 194 us, 26% of the measured copy rate;
// bf16 x 22528 174 us, 16%.
template <int XT, int YT>
__global__ void __launch_bounds__(kThreads) norm_long_kernel(const NormArgs a) {
    __shared__ float part[32];
    const int64_t t = blockIdx.x;
    const auto *x = row_of<XT>(a.x, a.nb_x, t);
    auto *y = row_of<YT>(a.y, a.nb_y, t);
    float s = 0.f;
    for (int64_t m = threadIdx.x; m < a.M; m += kThreads) s += to_float(x[m]);
    const float mean = block_sum(s, part) / static_cast<float>(a.M);
    s = 0.f;
    for (int64_t m = threadIdx.x; m < a.M; m += kThreads) {
        const float d = to_float(x[m]) - mean;
        s = fmaf(d, d, s);
    }
    const float rstd = 1.f / sqrtf(block_sum(s, part) / static_cast<float>(a.M) + a.eps);
    for (int64_t m = threadIdx.x; m < a.M; m += kThreads) {
        float v = (to_float(x[m]) - mean) * rstd;
        if (a.w) v *= load_any(a.w, a.w_type, m);
        if (a.b) v += load_any(a.b, a.w_type, m);
        y[m] = from_float<YT>(v);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[t] = mean;
        if (a.rstd) a.rstd[t] = rstd;
    }
}

struct NormBackArgs {
    const void *dy, *x, *w;
    const float *mean, *rstd;
    void *dx;
    float *dw, *db, *part;           // part: {M, slices, 2}, or NULL (no dw, no db)
    int64_t nb_dy, nb_x, nb_dx, M, T;
    int w_type;
    int width, groups, stages;       // threads per row, rows at once, rows staged per group
};

// The backward pass: dx, and this CTA's part of dw and db.  `width` threads share
// a row, 32 columns each; a CTA (one per SM) has `groups` rows in work and goes on
// to others until none is left, so the sums of a column stay with its thread.
// Each thread copies its pieces of the next rows into shared memory while this
// one is reduced: the loads never wait for a row's sums.  Two columns at a time
// in packed fp32 arithmetic: half the instructions, the same roundings.
//
// bf16, 16384 x 5120: 89 us, 5.7 TB/s (84% of the measured copy rate); a main pass of
// about 83 us in which the 15 warps that the registers allow issue in 50% of the
// cycles, waiting for shared memory and for the row's two sums, and 4 us for the
// sum of the CTAs' parts.  16 columns per thread (20 warps, w and the row in
// registers): 138 us, the reductions then are most of the work.  (A variant without the
// checks for a missing unit, for rows that fill every lane, keeps more of a row
// in flight than 128 registers hold, and is 35% slower.)
template <int XT, int DT, int E, int COLS>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_back_kernel(const NormBackArgs a) {
    using X = Staged<XT, E>;
    using D = Staged<DT, E>;
    using U = Units<E>;
    constexpr int kCount = COLS / U::kSize;
    extern __shared__ __align__(16) char sm[];
    let_next_start();
    const Place place(a.M, a.width), &p = place;
    float *ws = reinterpret_cast<float *>(sm);                       // w as floats
    float2 *red = reinterpret_cast<float2 *>(sm + p.width * COLS * 4);    // {2, 32}
    char *ring = reinterpret_cast<char *>(red + 64);
    const X xs(ring, p, a.x, a.nb_x, a.T, a.stages);
    const D ds(ring + xs.room(p, a.stages), p, a.dy, a.nb_dy, a.T, a.stages);
    const unsigned step = gridDim.x * a.groups, T = static_cast<unsigned>(a.T);
    const unsigned r0 = blockIdx.x * a.groups + p.group;
    // rows; all advance by `step`
    const int64_t up_x = step * a.nb_x, up_dy = step * a.nb_dy, up_dx = step * a.nb_dx;
    const char *x = static_cast<const char *>(a.x) + r0 * a.nb_x, *x_next = x;
    const char *dy = static_cast<const char *>(a.dy) + r0 * a.nb_dy, *dy_next = dy;
    char *dx = static_cast<char *>(a.dx) + r0 * a.nb_dx + p.lane * D::kBytes;
    const float *mean_at = a.mean + r0, *rstd_at = a.rstd + r0;
    unsigned t_next = r0;                            // (T <= 2^31, step <= 2432: no overflow)
    auto issue = [&](int st) {
        if (t_next < T) {
            xs.issue(x_next, st, p);
            ds.issue(dy_next, st, p);
        }
        commit_copies();
        t_next += step;
        x_next += up_x;
        dy_next += up_dy;
    };
    for (int s = 0; s + 1 < a.stages; ++s) issue(s);
    stage_params<E>(ws, a.w, a.w_type, 1.f, p.M, p.width);
    __syncthreads();

    uint64_t dw[kCount][U::kPairs], db[kCount][U::kPairs];
#pragma unroll
    for (int u = 0; u < kCount; ++u)
#pragma unroll
        for (int j = 0; j < U::kPairs; ++j) dw[u][j] = db[u][j] = 0;
    auto get_w = [&](int u, const Place &p, uint64_t (&w)[U::kPairs]) {
        if constexpr (E == 1) {
            const int m = p.column<E>(2 * u), n = p.column<E>(2 * u + 1);
            w[0] = ptx::pack2(ws[m], p.has<E>(2 * u + 1) ? ws[n] : 0.f);
        } else {
#pragma unroll
            for (int h = 0; h < E / 4; ++h) {
                const float4 q = *reinterpret_cast<const float4 *>(ws + ((u * (E / 4) + h) * p.width + p.lane) * 4);
                w[2 * h] = ptx::pack2(q.x, q.y);
                w[2 * h + 1] = ptx::pack2(q.z, q.w);
            }
        }
    };
    float mean_next = 0.f, rstd_next = 0.f;
    if (r0 < T) {
        mean_next = *mean_at;
        rstd_next = *rstd_at;
    }
    const float each = 1.f / static_cast<float>(p.M);
    int st = 0, odd = 0;
    for (unsigned t = r0; t < T; t += step) {
        if (E > 1) {
            issue(st == 0 ? a.stages - 1 : st - 1);
            wait_copies(a.stages - 1);
        } else {
            // every thread's copies of this row have to be there, and every thread
            // be done with the row before it, which the next copies overwrite
            wait_copies(a.stages - 2);
            if (p.warps > 1) asm volatile("bar.sync %0, %1;" ::"r"(p.group + 1), "r"(p.width) : "memory");
            else __syncwarp();
            issue(st == 0 ? a.stages - 1 : st - 1);
        }
        // the places of up to 24 singles are cheaper to find again for every row
        // than to keep in registers
        Place p = place;
        if (E == 1) asm volatile("" : "+r"(p.width));
        const uint64_t mean = both(mean_next), rstd = both(rstd_next);
        mean_at += step;
        rstd_at += step;
        if (t + step < T) {
            mean_next = *mean_at;
            rstd_next = *rstd_at;
        }
        uint64_t sg = 0, sgx = 0;
#pragma unroll
        for (int u = 0; u < kCount; ++u) {
            if (!has_unit<E>(u, p)) continue;
            uint64_t w[U::kPairs], d[U::kPairs], xh[U::kPairs];
            get_w(u, p, w);
            xs.get(u, st, x, p, xh);
            ds.get(u, st, dy, p, d);
#pragma unroll
            for (int j = 0; j < U::kPairs; ++j) {
                xh[j] = ptx::mul2(ptx::sub2(xh[j], mean), rstd);
                const uint64_t g = ptx::mul2(d[j], w[j]);
                sg = ptx::add2(sg, g);
                sgx = ptx::fma2(g, xh[j], sgx);
                dw[u][j] = ptx::fma2(d[j], xh[j], dw[u][j]);
                db[u][j] = ptx::add2(db[u][j], d[j]);
            }
        }
        float2 sum = make_float2(warp_sum(add_halves(sg)), warp_sum(add_halves(sgx)));
        if (p.warps > 1) {
            sum = exchange(sum, p, red, odd);
            sum = make_float2(warp_sum(sum.x), warp_sum(sum.y));
        }
        float r, unused;
        ptx::unpack2(rstd, r, unused);
        // dx = rstd * (g + (x - mean) * slope + level).  rstd stays outside, as its square
        // may be no float: it overflows for rows whose spread is below 5e-20, and
        // loses digits above 1e18.
        const uint64_t slope = both(-r * (sum.y * each)), level = both(-(sum.x * each));
#pragma unroll
        for (int u = 0; u < kCount; ++u) {
            if (!has_unit<E>(u, p)) continue;
            // read again: the registers that would keep g and xh hold dw and db
            uint64_t w[U::kPairs], xh[U::kPairs], g[U::kPairs];
            get_w(u, p, w);
            xs.get(u, st, x, p, xh);
            ds.get(u, st, dy, p, g);
#pragma unroll
            for (int j = 0; j < U::kPairs; ++j) {
                const uint64_t rest = ptx::fma2(ptx::sub2(xh[j], mean), slope, level);
                g[j] = ptx::mul2(ptx::fma2(g[j], w[j], rest), rstd);
            }
            put_unit<DT, E>(dx, u, p, g);
        }
        st = st + 1 == a.stages ? 0 : st + 1;
        x += up_x;
        dy += up_dy;
        dx += up_dx;
    }
    if (!a.part) return;
    float *out_w = a.part + static_cast<int64_t>(blockIdx.x) * p.M;
    float *out_b = out_w + static_cast<int64_t>(gridDim.x) * p.M;
    if (E > 1 && a.groups == 1) {
#pragma unroll
        for (int u = 0; u < kCount; ++u) {
            if (!has_unit<E>(u, p)) continue;
            put_floats<U::kPairs>(out_w + p.column<E>(u), dw[u]);
            put_floats<U::kPairs>(out_b + p.column<E>(u), db[u]);
        }
        return;
    }
    // the groups' sums in shared memory ({groups, 2, pairs, width}), then every group
    // adds up a share of the pairs over all groups, in order
    wait_copies(0);
    __syncthreads();
    constexpr int kAll = kCount * U::kPairs;
    uint64_t *all = reinterpret_cast<uint64_t *>(ring) + p.lane;
    const int of_group = 2 * kAll * p.width;
#pragma unroll
    for (int u = 0; u < kCount; ++u) {
#pragma unroll
        for (int j = 0; j < U::kPairs; ++j) {
            all[p.group * of_group + (u * U::kPairs + j) * p.width] = dw[u][j];
            all[p.group * of_group + (kAll + u * U::kPairs + j) * p.width] = db[u][j];
        }
    }
    __syncthreads();
    for (int k = p.group; k < 2 * kAll; k += a.groups) {
        uint64_t sum = all[k * p.width];
        for (int g = 1; g < a.groups; ++g) sum = ptx::add2(sum, all[g * of_group + k * p.width]);
        float *out = k < kAll ? out_w : out_b;
        const int u = k % kAll / U::kPairs, j = k % U::kPairs;
        const int m = E == 1 ? p.column<E>(2 * u) : p.column<E>(u) + 2 * j;
        const int n = E == 1 ? p.column<E>(2 * u + 1) : m + 1;
        float lo, hi;
        ptx::unpack2(sum, lo, hi);
        if (m < p.M) out[m] = lo;
        if (n < p.M) out[n] = hi;
    }
}

// Rows of more columns than 512 threads hold, or unaligned ones of which no two fit
// in shared memory: the columns' sums, then dx from one CTA per row.  2048 rows, f32
// x 20480: 273 us, 27% of the measured copy rate; bf16: 200 us, 19%.
template <int XT, int DT>
__global__ void __launch_bounds__(kThreads) norm_back_row_kernel(const NormBackArgs a) {
    __shared__ float part[32];
    const int64_t t = blockIdx.x;
    const auto *x = row_of<XT>(a.x, a.nb_x, t);
    const auto *dy = row_of<DT>(a.dy, a.nb_dy, t);
    auto *dx = row_of<DT>(a.dx, a.nb_dx, t);
    const float mean = a.mean[t], rstd = a.rstd[t];
    float sg = 0.f, sgx = 0.f;
    for (int64_t m = threadIdx.x; m < a.M; m += kThreads) {
        const float g = to_float(dy[m]) * (a.w ? load_any(a.w, a.w_type, m) : 1.f);
        sg += g;
        sgx = fmaf(g, (to_float(x[m]) - mean) * rstd, sgx);
    }
    const float mg = block_sum(sg, part) / static_cast<float>(a.M);
    const float mgx = block_sum(sgx, part) / static_cast<float>(a.M);
    for (int64_t m = threadIdx.x; m < a.M; m += kThreads) {
        const float g = to_float(dy[m]) * (a.w ? load_any(a.w, a.w_type, m) : 1.f);
        const float xh = (to_float(x[m]) - mean) * rstd;
        dx[m] = from_float<DT>(rstd * (g - mg - xh * mgx));
    }
}

// Column sums over one slice of rows, into the workspace: {M, slices, 2}.
template <int XT, int DT>
__global__ void __launch_bounds__(kThreads) norm_back_cols_kernel(const NormBackArgs a) {
    const int64_t m = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (m >= a.M) return;
    const int64_t t0 = a.T * blockIdx.y / gridDim.y, t1 = a.T * (blockIdx.y + 1) / gridDim.y;
    float sw = 0.f, sb = 0.f;
    for (int64_t t = t0; t < t1; ++t) {
        const float d = to_float(row_of<DT>(a.dy, a.nb_dy, t)[m]);
        sw = fmaf(d, (to_float(row_of<XT>(a.x, a.nb_x, t)[m]) - a.mean[t]) * a.rstd[t], sw);
        sb += d;
    }
    a.part[blockIdx.y * a.M + m] = sw;
    a.part[(gridDim.y + blockIdx.y) * a.M + m] = sb;
}

// A CTA sums 32 columns of dw (blockIdx.y 0) or db over the slices: eight warps
// take every eighth.
__global__ void __launch_bounds__(kThreads) norm_back_join_kernel(const float *part, int slices,
                                                                  int64_t M, float *dw, float *db) {
    __shared__ float sums[kThreads / 32][32];
    wait_previous();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float *out = blockIdx.y == 0 ? dw : db;
    if (!out) return;
    part += static_cast<int64_t>(blockIdx.y) * slices * M + m;
    float s = 0.f;
    constexpr int kMost = static_cast<int>(kSlices) / (kThreads / 32);
    float v[kMost];                                  // every load before the first sum
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
        const int k = warp + j * (kThreads / 32);
        v[j] = m < M && k < slices ? __ldcg(part + k * M) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kMost; ++j) s += v[j];
    sums[warp][lane] = s;
    __syncthreads();
    if (warp > 0 || m >= M) return;
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) s += sums[w][lane];
    out[m] = s;
}

// Threads that share a row.
int width_of(int64_t M, int cols) { return static_cast<int>((M + 32 * cols - 1) / (32 * cols)) * 32; }

int64_t slices_of(int64_t T) { return T < kSlices ? T : kSlices; }

// Shares a CTA among rows: width, groups and stages of the backward kernel, with
// `fixed` bytes of shared memory besides the staged rows of `row_bytes` each.  As
// many rows at once as fit, twice if they can be (one in work, one on its way),
// but no CTA with many rows while others have none.  Named barriers 1 .. 15 are
// the groups' (a warp that has a row alone needs none).
void share_cta(NormBackArgs &a, int cols, int fixed, int row_bytes) {
    a.width = width_of(a.M, cols);
    const int slots = (kSmem - fixed) / row_bytes;
    a.groups = static_cast<int>(std::min<int64_t>({kMaxThreads / a.width, a.width == 32 ? 16 : 15,
                                                   std::max(1, slots / 2), (a.T + kSlices - 1) / kSlices}));
    a.stages = std::max(1, std::min(kMaxStages, slots / a.groups));
}

template <int XT, int YT, int E, int NV>
cudaError_t launch_norm_few(const NormArgs &a, cudaStream_t st) {
    const int threads = std::max(a.width, 128 / a.width * a.width);
    const int64_t rows = threads / a.width;
    const auto kern = int64_t(a.pieces) * a.width * E == a.M ? norm_kernel<XT, YT, E, NV, true>
                                                             : norm_kernel<XT, YT, E, NV, false>;
    kern<<<static_cast<unsigned>((a.T + rows - 1) / rows), threads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int XT, int YT, int E, int NV, bool FULL>
cudaError_t launch_norm_many(const NormArgs &a, int fixed, cudaStream_t st) {
    const int threads = a.width * a.groups, smem = fixed + threads * a.pieces * E * plain_size(XT);
    const cudaError_t e = allow_smem<norm_many_kernel<XT, YT, E, NV, FULL>>();
    if (e != cudaSuccess) return e;
    norm_many_kernel<XT, YT, E, NV, FULL>
        <<<static_cast<unsigned>(std::min(kSlices, (a.T + a.groups - 1) / a.groups)), threads, smem, st>>>(a);
    return cudaGetLastError();
}

template <int XT, int YT, int E, int NV>
cudaError_t launch_norm_many(const NormArgs &a, int fixed, cudaStream_t st) {
    return int64_t(a.pieces) * a.width * E == a.M ? launch_norm_many<XT, YT, E, NV, true>(a, fixed, st)
                                                  : launch_norm_many<XT, YT, E, NV, false>(a, fixed, st);
}

// Fewer rows than the SMs have warps for are spread over more threads each, for
// latency.
constexpr int64_t kFewRows = 152 * 8;

template <int XT, int YT>
cudaError_t launch_norm(NormArgs a, bool wide, cudaStream_t st) {
    // 16 bytes of the narrower type, so that neither side moves less
    constexpr int E = plain_size(XT) == 2 && plain_size(YT) == 2 ? 8 : 4;
    const int64_t units = wide ? a.M / E : a.M;
    // threads per row: the fewest that hold it in so many pieces, in whole warps
    auto fits = [&](int pieces, int threads) {
        const int64_t width = (units + 32 * pieces - 1) / (32 * pieces) * 32;
        if (width > threads) return false;
        a.width = static_cast<int>(width);
        a.pieces = static_cast<int>((units + width - 1) / width);
        return true;
    };
    if (wide) {
        if (a.T < kFewRows && fits(4, 1024)) return launch_norm_few<XT, YT, E, 4>(a, st);
        // pieces per thread: 20, and fewer where shared memory holds so few rows that
        // half of the threads would be left over (2048 rows of 13312 bf16: 60 us
        // against 76 with 20 alone, before w and b were loaded four at a time, 35 us
        // since; rows of 5120 take 20 either way)
        NormArgs found = a;
        int fixed = 0;
        found.groups = 0;
        for (int pieces : {20, 10, 5}) {
            if (!fits(pieces, kMaxThreads)) break;
            const int row = a.pieces * a.width * E, besides = 256 + 2 * row * 4;
            a.groups = std::min({kMaxThreads / a.width, a.width == 32 ? 16 : 15,
                                 (kSmem - besides) / (row * plain_size(XT))});
            if (a.groups < 1) break;
            found = a;
            fixed = besides;
            if (2 * a.groups * a.width > kMaxThreads) break;
        }
        if (found.groups > 0 && found.pieces <= 10) return launch_norm_many<XT, YT, E, 10>(found, fixed, st);
        if (found.groups > 0) return launch_norm_many<XT, YT, E, 20>(found, fixed, st);
    } else {
        if (a.T < kFewRows && fits(16, 1024)) return launch_norm_few<XT, YT, 1, 16>(a, st);
        // as many rows as fit twice, and as many threads for each as that leaves
        const int64_t room = row_room(a.M, plain_size(XT)), fixed = 256 + a.M * 8;
        if (a.M <= 128 * kMaxThreads && fixed + 2 * room <= kSmem) {
            a.width = width_of(a.M, 128);
            a.groups = static_cast<int>(std::min<int64_t>({kMaxThreads / a.width, a.width == 32 ? 16 : 15,
                                                           (kSmem - fixed) / (2 * room)}));
            if (a.groups < 16) a.width = std::max(a.width, kMaxThreads / a.groups / 32 * 32);
            const cudaError_t e = allow_smem<norm_odd_kernel<XT, YT>>();
            if (e != cudaSuccess) return e;
            norm_odd_kernel<XT, YT>
                <<<static_cast<unsigned>(std::min(kSlices, (a.T + a.groups - 1) / a.groups)), a.width * a.groups,
                   fixed + a.groups * 2 * room, st>>>(a);
            return cudaGetLastError();
        }
    }
    norm_long_kernel<XT, YT><<<static_cast<unsigned>(a.T), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int XT>
cudaError_t launch_norm(const NormArgs &a, int yt, bool wide, cudaStream_t st) {
    switch (yt) {
    case OOP_TYPE_F32: return launch_norm<XT, OOP_TYPE_F32>(a, wide, st);
    case OOP_TYPE_F16: return launch_norm<XT, OOP_TYPE_F16>(a, wide, st);
    default: return launch_norm<XT, OOP_TYPE_BF16>(a, wide, st);
    }
}

template <int XT, int DT>
cudaError_t join_slices(const NormBackArgs &a, int slices, cudaStream_t st) {
    return launch_dependent(norm_back_join_kernel, dim3(static_cast<unsigned>((a.M + 31) / 32), 2),
                            kThreads, 0, st, a.part, slices, a.M, a.dw, a.db);
}

// cudaErrorNotSupported: no room for two stages of a row of singles.
template <int XT, int DT, int E, int COLS>
cudaError_t launch_back_kernel(NormBackArgs a, cudaStream_t st) {
    const int width = width_of(a.M, COLS), fixed = width * COLS * 4 + 64 * 8;
    const int row = E == 1 ? row_room(a.M, plain_size(XT)) + row_room(a.M, plain_size(DT))
                           : width * COLS * (plain_size(XT) + plain_size(DT));
    share_cta(a, COLS, fixed, row);
    if (E == 1 && (a.stages < 2 || fixed + a.groups * 2 * row > kSmem)) return cudaErrorNotSupported;
    const int threads = a.width * a.groups;
    const int slices = static_cast<int>(std::min(kSlices, (a.T + a.groups - 1) / a.groups));
    const int ring = std::max(a.stages * a.groups * row, a.groups > 1 || E == 1 ? threads * COLS * 8 : 0);
    cudaError_t e = allow_smem<norm_back_kernel<XT, DT, E, COLS>>();
    if (e != cudaSuccess) return e;
    norm_back_kernel<XT, DT, E, COLS><<<slices, threads, fixed + ring, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess || !a.part) return e;
    return join_slices<XT, DT>(a, slices, st);
}

template <int XT, int DT>
cudaError_t launch_back(const NormBackArgs &a, bool wide, cudaStream_t st) {
    constexpr int E = plain_size(XT) == 2 && plain_size(DT) == 2 ? 8 : 4;
    constexpr int kSingles = kCols * 3 / 4;                  // columns of a thread, unaligned
    if (a.M <= kMaxThreads * (wide ? kCols : kSingles)) {
        g_kernel_launches = a.part ? 2 : 1;
        // singles: half the columns per thread while two rows' threads fit, then three
        // quarters (bf16, 4096 rows of 4097: 55 us; half, with one row at a time, 70)
        const bool half = 2 * width_of(a.M, kCols / 2) <= kMaxThreads;
        const cudaError_t e = wide   ? launch_back_kernel<XT, DT, E, kCols>(a, st)
                              : half ? launch_back_kernel<XT, DT, 1, kCols / 2>(a, st)
                                     : launch_back_kernel<XT, DT, 1, kSingles>(a, st);
        if (e != cudaErrorNotSupported) return e;
    }
    g_kernel_launches = a.part ? 3 : 1;
    if (a.part) {                        // first: dx may be written over dy
        const int64_t tiles = (a.M + kThreads - 1) / kThreads, slices = slices_of(a.T);
        norm_back_cols_kernel<XT, DT>
            <<<dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(slices)), kThreads, 0, st>>>(a);
        cudaError_t e = cudaGetLastError();
        if (e == cudaSuccess) e = join_slices<XT, DT>(a, static_cast<int>(slices), st);
        if (e != cudaSuccess) return e;
    }
    norm_back_row_kernel<XT, DT><<<static_cast<unsigned>(a.T), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

int check_norm(const int64_t ne[2]) {
    if (!ne) return OOP_ERR_NULL;
    const int rc = check_extent(ne[0], ne[1]);
    if (rc != OOP_OK) return rc;
    if (ne[0] == 0 && ne[1] > 0) return OOP_ERR_SHAPE;       // the mean of nothing
    if (ne[0] > 0x7fffffffLL || ne[1] > 0x7fffffffLL) return OOP_ERR_SHAPE;
    return OOP_OK;
}

}  // namespace
}  // namespace oop

using namespace oop;

extern "C" {

int oop_layer_norm(const void *x, int x_type, int64_t nb_x, const void *w, const void *b,
                   int w_type, void *y, int y_type, int64_t nb_y, float *mean, float *rstd,
                   const int64_t ne[2], float eps, void *stream) {
    g_kernel_launches = 0;
    int rc = check_norm(ne);
    if (rc != OOP_OK) return rc;
    const int64_t M = ne[0], T = ne[1];
    const int sx = plain_size(x_type), sy = plain_size(y_type), sw = plain_size(w_type);
    if (!sx || !sy || ((w || b) && !sw)) return OOP_ERR_TYPE;
    if (!(eps >= 0.f) || std::isinf(eps)) return OOP_ERR_VALUE;
    if ((rc = check_row_stride(M * sx, T, nb_x, sx, false)) != OOP_OK) return rc;
    if ((rc = check_row_stride(M * sy, T, nb_y, sy, true)) != OOP_OK) return rc;
    if (T == 0) return OOP_OK;
    if ((rc = check_pointer(x, sx)) != OOP_OK) return rc;
    if ((rc = check_pointer(y, sy)) != OOP_OK) return rc;
    if ((w && !is_aligned(w, sw)) || (b && !is_aligned(b, sw)) || !is_aligned(mean, 4) ||
        !is_aligned(rstd, 4))
        return OOP_ERR_ALIGN;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    const NormArgs a = {x, w, b, y, mean, rstd, nb_x, nb_y, M, T, w_type, 0, 0, 0, eps};
    const bool wide = M % 8 == 0 && is_aligned(x, 16) && is_aligned(y, 16) && (!w || is_aligned(w, 8 * sw)) &&
                      (!b || is_aligned(b, 8 * sw)) && nb_x % 16 == 0 && nb_y % 16 == 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = x_type == OOP_TYPE_F32   ? launch_norm<OOP_TYPE_F32>(a, y_type, wide, st)
                          : x_type == OOP_TYPE_F16 ? launch_norm<OOP_TYPE_F16>(a, y_type, wide, st)
                                                   : launch_norm<OOP_TYPE_BF16>(a, y_type, wide, st);
    if (e == cudaSuccess) g_kernel_launches = 1;
    return cuda_status(e);
}

size_t oop_layer_norm_back_workspace_size(const int64_t ne[2]) {
    if (check_norm(ne) != OOP_OK) return 0;
    return static_cast<size_t>(slices_of(ne[1]) * ne[0]) * 2 * sizeof(float);
}

int oop_layer_norm_back(const void *dy, int dy_type, int64_t nb_dy, const void *x, int x_type,
                        int64_t nb_x, const float *mean, const float *rstd, const void *w,
                        int w_type, void *dx, int64_t nb_dx, float *dw, float *db,
                        const int64_t ne[2], void *workspace, size_t workspace_bytes,
                        void *stream) {
    g_kernel_launches = 0;
    int rc = check_norm(ne);
    if (rc != OOP_OK) return rc;
    const int64_t M = ne[0], T = ne[1];
    const int sx = plain_size(x_type), sd = plain_size(dy_type), sw = plain_size(w_type);
    if (!sx || !gradient_type(dy_type) || (w && !sw)) return OOP_ERR_TYPE;
    if ((rc = check_row_stride(M * sx, T, nb_x, sx, false)) != OOP_OK) return rc;
    if ((rc = check_row_stride(M * sd, T, nb_dy, sd, false)) != OOP_OK) return rc;
    if ((rc = check_row_stride(M * sd, T, nb_dx, sd, true)) != OOP_OK) return rc;
    if (!is_aligned(dw, 4) || !is_aligned(db, 4) || (w && !is_aligned(w, sw))) return OOP_ERR_ALIGN;
    if (M == 0) return OOP_OK;
    int *status = nullptr;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {                                            // empty sums
        if ((rc = device_status_word(&status)) != OOP_OK) return rc;
        cudaError_t e = cudaSuccess;
        if (dw) e = cudaMemsetAsync(dw, 0, static_cast<size_t>(M) * 4, st);
        if (db && e == cudaSuccess) e = cudaMemsetAsync(db, 0, static_cast<size_t>(M) * 4, st);
        return cuda_status(e);
    }
    if ((rc = check_pointer(x, sx)) != OOP_OK) return rc;
    if ((rc = check_pointer(dy, sd)) != OOP_OK) return rc;
    if ((rc = check_pointer(dx, sd)) != OOP_OK) return rc;
    if ((rc = check_pointer(mean, 4)) != OOP_OK) return rc;
    if ((rc = check_pointer(rstd, 4)) != OOP_OK) return rc;
    const bool cols = dw || db;
    if (cols && (!workspace || workspace_bytes < oop_layer_norm_back_workspace_size(ne) ||
                 !is_aligned(workspace, 256)))
        return OOP_ERR_WORKSPACE;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    NormBackArgs a = {};
    a.dy = dy;
    a.x = x;
    a.w = w;
    a.mean = mean;
    a.rstd = rstd;
    a.dx = dx;
    a.dw = dw;
    a.db = db;
    a.part = cols ? static_cast<float *>(workspace) : nullptr;
    a.nb_dy = nb_dy;
    a.nb_x = nb_x;
    a.nb_dx = nb_dx;
    a.M = M;
    a.T = T;
    a.w_type = w_type;
    const bool wide = M % 8 == 0 && is_aligned(dy, 16) && is_aligned(x, 16) && is_aligned(dx, 16) &&
                      (!w || is_aligned(w, 8 * sw)) && nb_dy % 16 == 0 && nb_x % 16 == 0 && nb_dx % 16 == 0;
    const bool f32 = dy_type == OOP_TYPE_F32;
    cudaError_t e = cudaSuccess;
    switch (x_type) {
    case OOP_TYPE_F32:
        e = f32 ? launch_back<OOP_TYPE_F32, OOP_TYPE_F32>(a, wide, st)
                : launch_back<OOP_TYPE_F32, OOP_TYPE_BF16>(a, wide, st);
        break;
    case OOP_TYPE_F16:
        e = f32 ? launch_back<OOP_TYPE_F16, OOP_TYPE_F32>(a, wide, st)
                : launch_back<OOP_TYPE_F16, OOP_TYPE_BF16>(a, wide, st);
        break;
    default:
        e = f32 ? launch_back<OOP_TYPE_BF16, OOP_TYPE_F32>(a, wide, st)
                : launch_back<OOP_TYPE_BF16, OOP_TYPE_BF16>(a, wide, st);
    }
    if (e != cudaSuccess) g_kernel_launches = 0;
    return cuda_status(e);
}

}  // extern "C"
