// products.cu -- see products.cuh.
#include "products.cuh"

#include <algorithm>

#include "quant.cuh"

namespace oop {
namespace {

template <int TYPE>
__global__ void to_f32_kernel(const char *src, int64_t nb, int64_t cols, int64_t rows, float *dst, int64_t pitch) {
    using F = QFormat<TYPE>;
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < rows * cols; i += gridDim.x * 256LL) {
        const int64_t r = i / cols, c = i - r * cols;
        const uint8_t *row = reinterpret_cast<const uint8_t *>(src + r * nb);
        dst[r * pitch + c] = decode<TYPE>(row + c / F::QK * F::BYTES, static_cast<int>(c % F::QK));
    }
}

constexpr int kTile = 64, kDepth = 16;

__global__ void __launch_bounds__(256) product_kernel(const Product p) {
    __shared__ float as[kDepth][kTile + 1], bs[kDepth][kTile + 1];
    const int64_t tiles_n = (p.N + kTile - 1) / kTile;
    const int64_t m0 = blockIdx.x / tiles_n * kTile, n0 = blockIdx.x % tiles_n * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (int64_t z = blockIdx.y; z < p.batch; z += gridDim.y) {
        const float *a = p.a + z * p.a_mat, *b = p.b + z * p.b_mat;
        float acc[4][4] = {};
        for (int64_t k0 = 0; k0 < p.K; k0 += kDepth) {
            for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
                const int fast_a = p.a_col == 1, fast_b = p.b_col == 1;
                const int ka = fast_a ? i % kDepth : i / kTile, ma = fast_a ? i / kDepth : i % kTile;
                const int kb = fast_b ? i % kDepth : i / kTile, nb = fast_b ? i / kDepth : i % kTile;
                as[ka][ma] = m0 + ma < p.M && k0 + ka < p.K ? a[(m0 + ma) * p.a_row + (k0 + ka) * p.a_col] : 0.f;
                bs[kb][nb] = n0 + nb < p.N && k0 + kb < p.K ? b[(n0 + nb) * p.b_row + (k0 + kb) * p.b_col] : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kDepth; ++k) {
                float av[4], bv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    av[i] = as[k][ty + 16 * i];
                    bv[i] = bs[k][tx + 16 * i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                if (m >= p.M || n >= p.N) continue;
                float *c = p.c + z * p.c_mat + m * p.c_row + n;
                *c = p.beta == 0.f ? p.alpha * acc[i][j] : fmaf(p.beta, *c, p.alpha * acc[i][j]);
            }
    }
}

}  // namespace

cudaError_t launch_to_f32(const void *src, int type, int64_t nb, int64_t cols, int64_t rows, float *dst,
                          int64_t pitch, cudaStream_t st) {
    if (cols == 0 || rows == 0) return cudaSuccess;
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((rows * cols + 255) / 256, 1 << 20));
    const char *s = static_cast<const char *>(src);
#define OOP_CASE(T) \
    case T: to_f32_kernel<T><<<blocks, 256, 0, st>>>(s, nb, cols, rows, dst, pitch); break;
    switch (type) {
        OOP_CASE(OOP_TYPE_F32) OOP_CASE(OOP_TYPE_F16) OOP_CASE(OOP_TYPE_BF16) OOP_CASE(OOP_TYPE_Q4_0)
        OOP_CASE(OOP_TYPE_Q4_1) OOP_CASE(OOP_TYPE_Q5_0) OOP_CASE(OOP_TYPE_Q5_1) OOP_CASE(OOP_TYPE_Q8_0)
        OOP_CASE(OOP_TYPE_Q2_K) OOP_CASE(OOP_TYPE_Q3_K) OOP_CASE(OOP_TYPE_Q4_K) OOP_CASE(OOP_TYPE_Q5_K)
        OOP_CASE(OOP_TYPE_Q6_K)
    }
#undef OOP_CASE
    ++g_kernel_launches;
    return cudaGetLastError();
}

cudaError_t launch_product(const Product &p, cudaStream_t st) {
    if (p.M == 0 || p.N == 0 || p.batch == 0) return cudaSuccess;
    const int64_t tiles = ((p.M + kTile - 1) / kTile) * ((p.N + kTile - 1) / kTile);
    product_kernel<<<dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(std::min<int64_t>(p.batch, 65535))), 256,
                     0, st>>>(p);
    ++g_kernel_launches;
    return cudaGetLastError();
}

}  // namespace oop
