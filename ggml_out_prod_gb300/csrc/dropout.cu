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
#include <cmath>

#include "oop_internal.cuh"
#include "rows.cuh"

namespace oop {
namespace {

constexpr int kThreads = 256;

struct DropArgs {
    const void *x;
    void *y;
    int64_t nb_x, nb_y, M, T;
    uint32_t k0, k1, c2, c3;
    uint32_t drop;               // 0 .. 65536
    float scale;
};

__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                        uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
        const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(p1);
        c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// One thread per group of 8 columns.
template <int TYPE>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropArgs a) {
    const int64_t groups = (a.M + 7) / 8;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t t = i / groups, g = i - t * groups;
    if (t >= a.T) return;
    const uint4 w = philox(static_cast<uint32_t>(g), static_cast<uint32_t>(t), a.c2, a.c3, a.k0, a.k1);
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
    const auto *x = row_of<TYPE>(a.x, a.nb_x, t);
    auto *y = row_of<TYPE>(a.y, a.nb_y, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t m = g * 8 + j;
        if (m < a.M) {
            const uint32_t bits = (j & 1) ? r[j / 2] >> 16 : r[j / 2] & 0xffffu;
            y[m] = from_float<TYPE>(bits >= a.drop ? to_float(x[m]) * a.scale : 0.f);
        }
    }
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
    // the counter holds m / 8 and t in 32 bits each; CTAs ride grid.x
    const int64_t groups = (M + 7) / 8;
    if (groups > 0xffffffffLL || T > 0xffffffffLL) return OOP_ERR_SHAPE;
    if (static_cast<double>(groups) * static_cast<double>(T) > 256.0 * 2147483647.0)
        return OOP_ERR_SHAPE;
    if ((rc = check_row_stride(M * size, T, nb_x, size, false)) != OOP_OK) return rc;
    if ((rc = check_row_stride(M * size, T, nb_y, size, true)) != OOP_OK) return rc;
    if (M == 0 || T == 0) return OOP_OK;
    if ((rc = check_pointer(x, size)) != OOP_OK) return rc;
    if ((rc = check_pointer(y, size)) != OOP_OK) return rc;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    DropArgs a = {x, y, nb_x, nb_y, M, T, static_cast<uint32_t>(seed),
                  static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(offset),
                  static_cast<uint32_t>(offset >> 32), 0, 0.f};
    a.drop = static_cast<uint32_t>(std::nearbyint(p * 65536.0));
    a.scale = a.drop < 65536 ? static_cast<float>(65536.0 / (65536 - a.drop)) : 0.f;
    const auto kern = type == OOP_TYPE_F32   ? dropout_kernel<OOP_TYPE_F32>
                      : type == OOP_TYPE_F16 ? dropout_kernel<OOP_TYPE_F16>
                                             : dropout_kernel<OOP_TYPE_BF16>;
    kern<<<static_cast<unsigned>((groups * T + kThreads - 1) / kThreads), kThreads, 0,
           static_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) g_kernel_launches = 1;
    return cuda_status(e);
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
