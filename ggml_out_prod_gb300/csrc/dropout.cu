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
    const void *x;
    void *y;
    int64_t nb_x, nb_y, M;
    uint32_t t0, rows, groups;   // the launch's rows; groups of 8 columns per row
    uint64_t inverse;            // floor(2^64 / groups) + 1: i / groups = high half of i * inverse
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

// Group i of the launch: row and group of the row (i < 2^31 and groups < 2^32,
// so the truncated product is exact; one group per row needs no division).
__device__ __forceinline__ void place(uint32_t i, const DropArgs &a, uint32_t &t, uint32_t &g) {
    t = a.groups == 1 ? i : static_cast<uint32_t>(__umul64hi(i, a.inverse));
    g = i - t * a.groups;
}

// A thread takes G groups of 8 columns, whole and aligned (M % 8 == 0): all
// their loads are in flight while their masks are computed.
template <int TYPE, int G>
__global__ void __launch_bounds__(kThreads) dropout_wide_kernel(const DropArgs a) {
    constexpr int E = 16 / plain_size(TYPE), N = 8 / E;
    const uint32_t total = a.rows * a.groups;
    uint32_t t[G], g[G];
    Packed<TYPE, E> raw[G][N];
#pragma unroll
    for (int k = 0; k < G; ++k) {
        const uint32_t i = (blockIdx.x * G + k) * kThreads + threadIdx.x;
        place(i, a, t[k], g[k]);
        if (i < total && a.drop < 65536) {
            const auto *x = row_of<TYPE>(a.x, a.nb_x, int64_t(a.t0) + t[k]) + int64_t(g[k]) * 8;
#pragma unroll
            for (int n = 0; n < N; ++n) raw[k][n] = load_stream<TYPE, E>(x + n * E);
        }
    }
#pragma unroll
    for (int k = 0; k < G; ++k) {
        const uint32_t i = (blockIdx.x * G + k) * kThreads + threadIdx.x;
        if (i >= total) return;
        const uint32_t keep = a.drop < 65536 ? keep_bits(g[k], a.t0 + t[k], a) : 0u;
        auto *y = row_of<TYPE>(a.y, a.nb_y, int64_t(a.t0) + t[k]) + int64_t(g[k]) * 8;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float v[E];
            raw[k][n].get(v);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = (keep >> (n * E + e)) & 1u ? v[e] * a.scale : 0.f;
            store_stream<TYPE, E>(y + n * E, v);
        }
    }
}

// Rows of any alignment: a lane computes the mask of one group; then the warp
// goes over its 32 groups four at a time, a lane per element, so that
// neighbouring lanes touch neighbouring elements.
template <int TYPE>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropArgs a) {
    const uint32_t total = a.rows * a.groups, lane = threadIdx.x & 31;
    const uint32_t i0 = blockIdx.x * kThreads + (threadIdx.x & ~31u);     // the warp's first group
    typename Plain<TYPE>::S raw[8];
    int64_t at[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t i = i0 + 4 * k + lane / 8;
        uint32_t t, g;
        place(i, a, t, g);
        const int64_t m = int64_t(g) * 8 + lane % 8;
        at[k] = i < total && m < a.M ? (int64_t(a.t0) + t) * a.nb_y + m * plain_size(TYPE) : -1;
        if (at[k] >= 0 && a.drop < 65536) raw[k] = row_of<TYPE>(a.x, a.nb_x, int64_t(a.t0) + t)[m];
    }
    uint32_t t, g, keep = 0;
    place(i0 + lane, a, t, g);
    if (a.drop < 65536) keep = keep_bits(g, a.t0 + t, a);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t bits = __shfl_sync(0xffffffffu, keep, 4 * k + lane / 8);
        if (at[k] < 0) continue;
        const float v = (bits >> (lane % 8)) & 1u ? to_float(raw[k]) * a.scale : 0.f;
        *reinterpret_cast<typename Plain<TYPE>::S *>(static_cast<char *>(a.y) + at[k]) = from_float<TYPE>(v);
    }
}

template <int TYPE>
void launch_dropout(const DropArgs &a, bool wide, cudaStream_t st) {
    constexpr int G = TYPE == OOP_TYPE_F32 ? 2 : 4;        // 64 bytes per thread
    const int64_t total = int64_t(a.rows) * a.groups;
    if (wide)
        dropout_wide_kernel<TYPE, G>
            <<<static_cast<unsigned>((total + G * kThreads - 1) / (G * kThreads)), kThreads, 0, st>>>(a);
    else
        dropout_kernel<TYPE>
            <<<static_cast<unsigned>((total + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
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
    DropArgs a = {};
    a.x = x;
    a.y = y;
    a.nb_x = nb_x;
    a.nb_y = nb_y;
    a.M = M;
    a.groups = static_cast<uint32_t>(groups);
    a.inverse = ~uint64_t(0) / a.groups + 1;
    for (int i = 0; i < 10; ++i) {
        a.k0[i] = static_cast<uint32_t>(seed) + static_cast<uint32_t>(i) * 0x9E3779B9u;
        a.k1[i] = static_cast<uint32_t>(seed >> 32) + static_cast<uint32_t>(i) * 0xBB67AE85u;
    }
    a.c2 = static_cast<uint32_t>(offset);
    a.c3 = static_cast<uint32_t>(offset >> 32);
    a.drop = static_cast<uint32_t>(std::nearbyint(p * 65536.0));
    a.scale = a.drop < 65536 ? static_cast<float>(65536.0 / (65536 - a.drop)) : 0.f;
    const bool wide = M % 8 == 0 && is_aligned(x, 16) && is_aligned(y, 16) && nb_x % 16 == 0 &&
                      nb_y % 16 == 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t rows = std::min(T, kMaxGroups / groups);
    int launches = 0;
    for (int64_t t0 = 0; t0 < T; t0 += rows, ++launches) {
        a.t0 = static_cast<uint32_t>(t0);
        a.rows = static_cast<uint32_t>(std::min(rows, T - t0));
        if (type == OOP_TYPE_F32) launch_dropout<OOP_TYPE_F32>(a, wide, st);
        else if (type == OOP_TYPE_F16) launch_dropout<OOP_TYPE_F16>(a, wide, st);
        else launch_dropout<OOP_TYPE_BF16>(a, wide, st);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_status(e);
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
