// dropout.cu -- dropout whose mask is a function of position, never stored.
//
//   y[m, t] = r(m, t) >= D ? x[m, t] * 65536 / (65536 - D) : 0,
//   D = round(65536 * p)
//
// r is 16 bits of Philox4x32-10, the counter-based generator of Salmon, Moraes,
// Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3" (SC 2011): key =
// seed, counter = (m / 8, t, offset low, offset high).  One call gives four
// 32-bit words, so eight halves, one for each column of the group of 8 (the
// low half of a word first).  The backward pass is the same map on dy.  16
// bits halve the generator's work against one word per element; the scale is
// that of the rounded probability, so the mean of y is exactly x.
#include <algorithm>
#include <cmath>

#include "oop_internal.cuh"
#include "rows.cuh"

namespace oop {
namespace {

constexpr int kThreads = 256;

constexpr int64_t kMaxGroups = int64_t(1) << 31;     // of one launch: 32-bit group numbers

struct DropArgs {
    const void *x;               // the launch's first row
    void *y;
    int64_t nb_x, nb_y, M;
    uint32_t t0, rows, groups;   // the launch's rows; units of a row: groups of 8 columns, or spans of 256
    uint64_t inverse;            // floor(2^64 / groups) + 1: i / groups = high half of i * inverse
    uint32_t next_t, next_g;     // kThreads groups on: kThreads / groups rows and the rest
    bool dense;                  // x's and y's rows follow each other
    uint32_t k0[10], k1[10];     // the key of each round
    uint32_t c2, c3;
    uint32_t drop;               // 0 .. 65536
    float scale;
};

// The low and high product halves of a round come from one wide multiply each.
__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, const DropArgs &a) {
    uint32_t c2 = a.c2, c3 = a.c3;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
        const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ a.k0[i];
        c1 = static_cast<uint32_t>(p1);
        c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ a.k1[i];
        c3 = static_cast<uint32_t>(p0);
    }
    return make_uint4(c0, c1, c2, c3);
}

// Bit j: column j of the group stays.
__device__ __forceinline__ uint32_t keep_bits(uint32_t g, uint32_t t, const DropArgs &a) {
    if (a.drop == 0) return 0xffu;
    const uint4 w = philox(g, t, a);
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
    uint32_t keep = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        keep |= (r[j] & 0xffffu) >= a.drop ? 1u << (2 * j) : 0u;
        keep |= (r[j] >> 16) >= a.drop ? 2u << (2 * j) : 0u;
    }
    return keep;
}

// Unit i of the launch: row and unit of the row (i <= 2^31 and groups < 2^32, so
// the truncated product is exact; one unit per row needs no division).
__device__ __forceinline__ void place(uint32_t i, const DropArgs &a, uint32_t &t, uint32_t &g) {
    t = a.groups == 1 ? i : static_cast<uint32_t>(__umul64hi(i, a.inverse));
    g = i - t * a.groups;
}

// A thread takes G groups of 8 columns, whole and aligned (M % 8 == 0): all
// their loads are in flight while their masks are computed.  The generator
// bounds this kernel as much as memory does (20 wide multiplies and 20
// three-way logic operations for 8 elements), so what surrounds it is lean: one
// division for the G groups, addresses by addition, halves compared in place.
//
// bf16, 16384 x 9728: 103 us, 6.2 TB/s (91% of the measured copy rate), with 8 CTAs
// per SM; with the 5 that an unbounded register count leaves, 113 to 115 us.  64
// bytes per thread: the same there, 5.4 us against 4.2 for f32, 512 x 2560.
template <int TYPE, int G>
__global__ void __launch_bounds__(kThreads, 8) dropout_wide_kernel(const DropArgs a) {
    constexpr int E = 16 / plain_size(TYPE), N = 8 / E;
    const uint32_t total = a.rows * a.groups, first = blockIdx.x * (G * kThreads) + threadIdx.x;
    uint32_t t[G], g[G];
    Packed<TYPE, E> raw[G][N];
    place(first, a, t[0], g[0]);
#pragma unroll
    for (int k = 1; k < G; ++k) {
        t[k] = t[k - 1] + a.next_t;
        g[k] = g[k - 1] + a.next_g;
        if (g[k] >= a.groups) {
            g[k] -= a.groups;
            ++t[k];
        }
    }
    // byte offsets, of x and of y
    auto offset = [&](int k, int64_t nb) -> int64_t {
        if (a.dense) return int64_t(first + k * kThreads) * (8 * plain_size(TYPE));
        return int64_t(t[k]) * nb + int64_t(g[k]) * (8 * plain_size(TYPE));
    };
    if (a.drop < 65536) {
#pragma unroll
        for (int k = 0; k < G; ++k) {
            if (first + k * kThreads >= total) break;
            const char *x = static_cast<const char *>(a.x) + offset(k, a.nb_x);
#pragma unroll
            for (int n = 0; n < N; ++n)
                raw[k][n] = load_stream<TYPE, E>(reinterpret_cast<const typename Plain<TYPE>::S *>(x) + n * E);
        }
    }
    const uint32_t high = a.drop << 16;              // (drop < 65536)
#pragma unroll
    for (int k = 0; k < G; ++k) {
        if (first + k * kThreads >= total) return;
        float v[N][E];
        if (a.drop < 65536) {
            uint4 w = make_uint4(~0u, ~0u, ~0u, ~0u);
            if (a.drop > 0) w = philox(g[k], a.t0 + t[k], a);
            const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int n = 0; n < N; ++n) {
                raw[k][n].get(v[n]);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const uint32_t word = r[(n * E + e) / 2], half = (e & 1) ? word : word << 16;
                    v[n][e] = half >= high ? v[n][e] * a.scale : 0.f;
                }
            }
        } else {
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < E; ++e) v[n][e] = 0.f;
        }
        char *y = static_cast<char *>(a.y) + offset(k, a.nb_y);
#pragma unroll
        for (int n = 0; n < N; ++n)
            store_stream<TYPE, E>(reinterpret_cast<typename Plain<TYPE>::S *>(y) + n * E, v[n]);
    }
}

// Rows of any alignment.  A warp takes 256 columns of a row: each lane computes
// the mask of one of their 32 groups, then the lanes go over the columns side by
// side, E (1 or 2, as the rows' alignment allows) each, and fetch the bits from
// the lane that has them.
constexpr int kSpan = 256;

template <int TYPE, int E>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropArgs a) {
    constexpr int N = kSpan / (32 * E);
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);    // the warp's span
    uint32_t t, span;
    place(i, a, t, span);
    if (t >= a.rows) return;
    const int64_t m0 = int64_t(span) * kSpan + lane * E;
    const auto *x = row_of<TYPE>(a.x, a.nb_x, t) + m0;
    auto *y = row_of<TYPE>(a.y, a.nb_y, t) + m0;
    const int left = static_cast<int>(min(a.M - m0, int64_t(kSpan)));        // columns from this lane's first
    Packed<TYPE, E> raw[N];
    if (a.drop < 65536) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (k * 32 * E < left) raw[k] = load_stream<TYPE, E>(x + k * 32 * E);
    }
    const uint32_t keep = a.drop < 65536 ? keep_bits(span * 32 + lane, a.t0 + t, a) : 0u;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const uint32_t bits = __shfl_sync(0xffffffffu, keep, (k * 32 + lane) * E / 8) >> (lane * E % 8);
        if (k * 32 * E >= left) continue;
        float v[E];
        raw[k].get(v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = (bits >> e) & 1u ? v[e] * a.scale : 0.f;
        store_stream<TYPE, E>(y + k * 32 * E, v);
    }
}

template <int TYPE>
void launch_dropout(const DropArgs &a, int e, cudaStream_t st) {
    constexpr int G = TYPE == OOP_TYPE_F32 ? 1 : 2;        // 32 bytes per thread
    const int64_t total = int64_t(a.rows) * a.groups;
    auto grid = [](int64_t n, int64_t per) { return static_cast<unsigned>((n + per - 1) / per); };
    if (e == 8) dropout_wide_kernel<TYPE, G><<<grid(total, G * kThreads), kThreads, 0, st>>>(a);
    else if (e == 2) dropout_kernel<TYPE, 2><<<grid(total, kThreads / 32), kThreads, 0, st>>>(a);
    else dropout_kernel<TYPE, 1><<<grid(total, kThreads / 32), kThreads, 0, st>>>(a);
}

int run_dropout(const void *x, int type, int64_t nb_x, void *y, int64_t nb_y, const int64_t ne[2],
                double p, uint64_t seed, uint64_t offset, void *stream) {
    if (!ne) return OOP_ERR_NULL;
    int rc = check_extent(ne[0], ne[1]);
    if (rc != OOP_OK) return rc;
    const int64_t M = ne[0], T = ne[1];
    const int size = plain_size(type);
    if (!size) return OOP_ERR_TYPE;
    if (!(p >= 0.0 && p <= 1.0)) return OOP_ERR_VALUE;
    // the counter holds m / 8 and t in 32 bits each; a launch takes whole rows
    const int64_t groups = (M + 7) / 8;
    if (groups > kMaxGroups / 2 || T > 0xffffffffLL) return OOP_ERR_SHAPE;
    if ((rc = check_row_stride(M * size, T, nb_x, size, false)) != OOP_OK) return rc;
    if ((rc = check_row_stride(M * size, T, nb_y, size, true)) != OOP_OK) return rc;
    if (M == 0 || T == 0) return OOP_OK;
    if ((rc = check_pointer(x, size)) != OOP_OK) return rc;
    if ((rc = check_pointer(y, size)) != OOP_OK) return rc;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    // elements of one access: 16 bytes and whole groups, two, or one
    auto fits = [&](int e, int bytes) {
        return M % e == 0 && is_aligned(x, bytes) && is_aligned(y, bytes) && nb_x % bytes == 0 &&
               nb_y % bytes == 0;
    };
    const int e = fits(8, 16) ? 8 : fits(2, 2 * size) ? 2 : 1;
    DropArgs a = {};
    a.x = x;
    a.y = y;
    a.nb_x = nb_x;
    a.nb_y = nb_y;
    a.M = M;
    a.groups = static_cast<uint32_t>(e == 8 ? groups : (M + kSpan - 1) / kSpan);
    a.inverse = ~uint64_t(0) / a.groups + 1;
    a.next_t = kThreads / a.groups;
    a.next_g = kThreads % a.groups;
    a.dense = nb_x == M * size && nb_y == M * size;
    for (int i = 0; i < 10; ++i) {
        a.k0[i] = static_cast<uint32_t>(seed) + static_cast<uint32_t>(i) * 0x9E3779B9u;
        a.k1[i] = static_cast<uint32_t>(seed >> 32) + static_cast<uint32_t>(i) * 0xBB67AE85u;
    }
    a.c2 = static_cast<uint32_t>(offset);
    a.c3 = static_cast<uint32_t>(offset >> 32);
    a.drop = static_cast<uint32_t>(std::nearbyint(p * 65536.0));
    a.scale = a.drop < 65536 ? static_cast<float>(65536.0 / (65536 - a.drop)) : 0.f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t rows = std::min(T, kMaxGroups / a.groups);
    int launches = 0;
    for (int64_t t0 = 0; t0 < T; t0 += rows, ++launches) {
        a.t0 = static_cast<uint32_t>(t0);
        a.x = static_cast<const char *>(x) + t0 * nb_x;
        a.y = static_cast<char *>(y) + t0 * nb_y;
        a.rows = static_cast<uint32_t>(std::min(rows, T - t0));
        if (type == OOP_TYPE_F32) launch_dropout<OOP_TYPE_F32>(a, e, st);
        else if (type == OOP_TYPE_F16) launch_dropout<OOP_TYPE_F16>(a, e, st);
        else launch_dropout<OOP_TYPE_BF16>(a, e, st);
        const cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess) return cuda_status(err);
    }
    g_kernel_launches = launches;
    return OOP_OK;
}

}  // namespace
}  // namespace oop

extern "C" {

int oop_dropout(const void *x, int type, int64_t nb_x, void *y, int64_t nb_y, const int64_t ne[2],
                double p, uint64_t seed, uint64_t offset, void *stream) {
    oop::g_kernel_launches = 0;
    return oop::run_dropout(x, type, nb_x, y, nb_y, ne, p, seed, offset, stream);
}

int oop_dropout_back(const void *dy, int type, int64_t nb_dy, void *dx, int64_t nb_dx,
                     const int64_t ne[2], double p, uint64_t seed, uint64_t offset, void *stream) {
    oop::g_kernel_launches = 0;
    if (!oop::gradient_type(type)) return OOP_ERR_TYPE;
    return oop::run_dropout(dy, type, nb_dy, dx, nb_dx, ne, p, seed, offset, stream);
}

}  // extern "C"
