// orthogonalise.cu -- the update of a weight made nearly orthogonal by
// Newton-Schulz steps, as the Muon optimiser does it.
//
//   X_0 = x / (|x|_F + eps),  X <- a X + (b A + c A A) X,  A = X X'
//
// A is taken on the smaller side: with M > N, X <- X (a + b X'X + c (X'X)^2) is
// the same polynomial of the singular values.
#include <algorithm>
#include <cmath>

#include "oop_internal.cuh"
#include "products.cuh"
#include "rows.cuh"

namespace oop {
namespace {

constexpr int kMaxSteps = 64;
constexpr float kDefault[3] = {3.4445f, -4.7750f, 2.0315f};

// Sums of squares of one thread: those of large, ordinary and small magnitudes
// apart, scaled so that none over- or underflows.
struct Squares {
    float big = 0.f, mid = 0.f, small = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float m = fabsf(v);
        if (m > 0x1p50f) {
            const float s = v * 0x1p-70f;
            big = fmaf(s, s, big);
        } else if (m < 0x1p-40f) {
            const float s = v * 0x1p70f;
            small = fmaf(s, s, small);
        } else {
            mid = fmaf(v, v, mid);
        }
        if (m != m) mid += m;
    }
};

// 1 / (|x|_F + eps) of each matrix as two factors of moderate size, by one CTA.
__global__ void __launch_bounds__(1024) norm_kernel(const char *x, int type, int64_t nb_row, int64_t nb_mat, int64_t N,
                                                    int64_t M, float eps, float2 *inv) {
    __shared__ double part[32];
    const char *p = x + blockIdx.x * nb_mat;
    Squares s;
    for (int64_t i = threadIdx.x; i < M * N; i += 1024) {
        const int64_t r = i / N;
        s.add(load_any(p + r * nb_row, type, i - r * N));
    }
    const double sum = block_sum(static_cast<double>(s.big) * 0x1p140 + static_cast<double>(s.mid) +
                                     static_cast<double>(s.small) * 0x1p-140, part);
    if (threadIdx.x == 0) {
        int e;
        const double v = 1.0 / (sqrt(sum) + static_cast<double>(eps));
        const double m = frexp(v, &e);
        const bool fine = v <= 0x1p200;                    // not Inf (zeros and eps = 0) or NaN
        inv[blockIdx.x] = fine ? make_float2(static_cast<float>(ldexp(m, e / 2)), static_cast<float>(ldexp(1.0, e - e / 2)))
                               : make_float2(static_cast<float>(v), 1.f);
    }
}

__global__ void start_kernel(const char *x, int type, int64_t nb_row, int64_t nb_mat, int64_t N, int64_t M,
                             const float2 *inv, float *dst) {
    const float2 f = inv[blockIdx.y];
    const char *p = x + blockIdx.y * nb_mat;
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < M * N; i += gridDim.x * 256LL) {
        const int64_t r = i / N;
        dst[blockIdx.y * M * N + i] = load_any(p + r * nb_row, type, i - r * N) * f.x * f.y;
    }
}

// q = a I + b A + c AA over B matrices {n, n}; A in p, AA in q.
__global__ void polynomial_kernel(const float *p, float *q, int64_t n, float a, float b, float c) {
    const int64_t base = blockIdx.y * n * n;
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < n * n; i += gridDim.x * 256LL)
        q[base + i] = (i / n == i % n ? a : 0.f) + b * p[base + i] + c * q[base + i];
}

__global__ void finish_kernel(const float *src, char *y, int type, int64_t nb_row, int64_t nb_mat, int64_t N, int64_t M,
                              float scale) {
    char *p = y + blockIdx.y * nb_mat;
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < M * N; i += gridDim.x * 256LL) {
        const int64_t r = i / N, c = i - r * N;
        const float v = scale * src[blockIdx.y * M * N + i];
        if (type == OOP_TYPE_F32) row_of<OOP_TYPE_F32>(p, nb_row, r)[c] = v;
        else row_of<OOP_TYPE_BF16>(p, nb_row, r)[c] = __float2bfloat16_rn(v);
    }
}

int check_sizes(const int64_t ne[3]) {
    if (!ne) return OOP_ERR_NULL;
    if (ne[0] < 0 || ne[1] < 0 || ne[2] < 0) return OOP_ERR_SHAPE;
    if (ne[0] > 0x7fffffLL || ne[1] > 0x7fffffLL || ne[2] > 65535) return OOP_ERR_SHAPE;
    return OOP_OK;
}

int check_matrices(const int64_t nb[2], const int64_t ne[3], int size, bool output) {
    int rc = check_row_stride(ne[0] * size, ne[1], nb[0], size, output);
    if (rc != OOP_OK) return rc;
    const int64_t bytes = ne[1] ? (ne[1] - 1) * nb[0] + ne[0] * size : 0;
    return check_row_stride(bytes, ne[2], nb[1], size, output);
}

}  // namespace
}  // namespace oop

using namespace oop;

extern "C" {

size_t oop_orthogonalise_workspace_size(const int64_t ne[3]) {
    if (check_sizes(ne) != OOP_OK || ne[0] == 0 || ne[1] == 0 || ne[2] == 0) return 0;
    const int64_t n = std::min(ne[0], ne[1]);
    return static_cast<size_t>(ne[2] * 8 + 255) / 256 * 256 +
           static_cast<size_t>(ne[2]) * static_cast<size_t>(2 * ne[0] * ne[1] + 2 * n * n) * 4;
}

int oop_orthogonalise(const void *x, int x_type, const int64_t nb_x[2], void *y, int y_type, const int64_t nb_y[2],
                      const int64_t ne[3], int steps, const float *coefs, float eps, float scale, void *workspace,
                      size_t workspace_bytes, void *stream) {
    g_kernel_launches = 0;
    if (!nb_x || !nb_y) return OOP_ERR_NULL;
    int rc = check_sizes(ne);
    if (rc != OOP_OK) return rc;
    if (!gradient_type(x_type) || !gradient_type(y_type)) return OOP_ERR_TYPE;
    if (steps < 0 || steps > kMaxSteps || !(eps >= 0.f && std::isfinite(eps)) || !std::isfinite(scale)) return OOP_ERR_VALUE;
    for (int i = 0; coefs && i < 3 * steps; ++i)
        if (!std::isfinite(coefs[i])) return OOP_ERR_VALUE;
    const int xs = plain_size(x_type), ys = plain_size(y_type);
    if ((rc = check_matrices(nb_x, ne, xs, false)) != OOP_OK) return rc;
    if ((rc = check_matrices(nb_y, ne, ys, true)) != OOP_OK) return rc;
    const int64_t N = ne[0], M = ne[1], B = ne[2];
    if (N == 0 || M == 0 || B == 0) return OOP_OK;
    if ((rc = check_pointer(x, xs)) != OOP_OK) return rc;
    if ((rc = check_pointer(y, ys)) != OOP_OK) return rc;
    if (!workspace || workspace_bytes < oop_orthogonalise_workspace_size(ne) || !is_aligned(workspace, 256))
        return OOP_ERR_WORKSPACE;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t n = std::min(M, N);
    float2 *inv = static_cast<float2 *>(workspace);
    float *cur = reinterpret_cast<float *>(static_cast<char *>(workspace) + (B * 8 + 255) / 256 * 256);
    float *next = cur + B * M * N, *A = next + B * M * N, *Q = A + B * n * n;
    const char *xp = static_cast<const char *>(x);
    auto grid = [&](int64_t c) { return dim3(static_cast<unsigned>(std::min<int64_t>((c + 255) / 256, 4096)), static_cast<unsigned>(B)); };
    norm_kernel<<<static_cast<unsigned>(B), 1024, 0, st>>>(xp, x_type, nb_x[0], nb_x[1], N, M, eps, inv);
    start_kernel<<<grid(M * N), 256, 0, st>>>(xp, x_type, nb_x[0], nb_x[1], N, M, inv, cur);
    g_kernel_launches = 2;
    cudaError_t e = cudaGetLastError();
    for (int s = 0; s < steps && e == cudaSuccess; ++s) {
        const float *c = coefs ? coefs + 3 * s : kDefault;
        // A[i, j] = sum over the larger side
        const int64_t row = M <= N ? N : 1, col = M <= N ? 1 : N, deep = std::max(M, N);
        e = launch_product({cur, cur, A, n, n, deep, B, row, col, M * N, row, col, M * N, n, n * n, 1.f, 0.f}, st);
        if (e == cudaSuccess)
            e = launch_product({A, A, Q, n, n, n, B, n, 1, n * n, n, 1, n * n, n, n * n, 1.f, 0.f}, st);
        if (e != cudaSuccess) break;
        polynomial_kernel<<<grid(n * n), 256, 0, st>>>(A, Q, n, c[0], c[1], c[2]);
        ++g_kernel_launches;
        if (M <= N) e = launch_product({Q, cur, next, M, N, M, B, n, 1, n * n, 1, N, M * N, N, M * N, 1.f, 0.f}, st);
        else e = launch_product({cur, Q, next, M, N, N, B, N, 1, M * N, n, 1, n * n, N, M * N, 1.f, 0.f}, st);
        std::swap(cur, next);
    }
    if (e != cudaSuccess) return cuda_status(e);
    finish_kernel<<<grid(M * N), 256, 0, st>>>(cur, static_cast<char *>(y), y_type, nb_y[0], nb_y[1], N, M, scale);
    ++g_kernel_launches;
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
