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
#include "pair_product.cuh"
#include "rows.cuh"

namespace oop {
namespace {

constexpr int kMaxSteps = 64;
constexpr float kDefault[3] = {3.4445f, -4.7750f, 2.0315f};

// The matrices between the products are held as two binary16 planes, hi + lo, of a
// scaled value: 22 bits or more, as many as a product of three terms keeps.  The
// scales leave room for magnitudes of 8, 64 and 256 below binary16's largest, and keep
// the planes of a 4096 x 4096 matrix (X's elements are about 2^-12) out of its
// subnormals.  bfloat16 planes would need no scale, but three of them and six terms.
constexpr float kScaleX = 0x1p13f, kScaleA = 0x1p10f, kScaleQ = 0x1p8f;

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

// The parts that a matrix's sum of squares is taken in: of its size alone, so that a
// matrix gives the same bits in any batch.
int64_t parts_of(int64_t elements) { return std::min<int64_t>(592, (elements + 16383) / 16384); }

// A warp's unit of work: up to kSpan columns of a row.
constexpr int kSpan = 2048;

// Eight elements from column c, those from column N on 0.
__device__ __forceinline__ void load8(const char *row, int type, int64_t c, int64_t N, bool wide, float (&v)[8]) {
    if (wide && c + 8 <= N) {
        if (type == OOP_TYPE_F32) {
            float a[4], b[4];
            load_stream<OOP_TYPE_F32, 4>(reinterpret_cast<const float *>(row) + c).get(a);
            load_stream<OOP_TYPE_F32, 4>(reinterpret_cast<const float *>(row) + c + 4).get(b);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
        } else {
            load_stream<OOP_TYPE_BF16, 8>(reinterpret_cast<const __nv_bfloat16 *>(row) + c).get(v);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < N ? load_any(row, type, c + i) : 0.f;
}

// Sum of squares of one part of each matrix (blockIdx.y).
__global__ void __launch_bounds__(256) squares_kernel(const char *x, int type, int64_t nb_row, int64_t nb_mat, int64_t N,
                                                      int64_t M, bool wide, double *sums) {
    __shared__ double part[32];
    const char *p = x + blockIdx.y * nb_mat;
    const int64_t spans = (N + kSpan - 1) / kSpan;
    Squares s;
    for (int64_t i = blockIdx.x * 8LL + (threadIdx.x >> 5); i < M * spans; i += gridDim.x * 8LL) {
        const int64_t r = i / spans, c0 = (i - r * spans) * kSpan, end = min(N, c0 + kSpan);
#pragma unroll 4
        for (int64_t c = c0 + (threadIdx.x & 31) * 8; c < end; c += 256) {
            float v[8];
            load8(p + r * nb_row, type, c, N, wide, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) s.add(v[k]);
        }
    }
    const double sum = block_sum(static_cast<double>(s.big) * 0x1p140 + static_cast<double>(s.mid) +
                                     static_cast<double>(s.small) * 0x1p-140, part);
    if (threadIdx.x == 0) sums[blockIdx.y * gridDim.x + blockIdx.x] = sum;
}

// 1 / (|x|_F + eps) as two factors of moderate size, by the first warp; NaN where a value is not finite.
__device__ __forceinline__ float2 inverse_norm(const double *sums, int parts, float eps) {
    double sum = 0.0;
    for (int i = threadIdx.x & 31; i < parts; i += 32) sum += sums[i];
    sum = warp_sum(sum);
    const double v = 1.0 / (sqrt(sum) + static_cast<double>(eps));
    if (!(sum <= 0x1p1000)) return make_float2(__int_as_float(0x7fc00000), 1.f);
    if (!(v <= 0x1p300)) return make_float2(static_cast<float>(v), 1.f);       // zeros and eps = 0
    int e;
    const double m = frexp(v, &e);
    return make_float2(static_cast<float>(ldexp(m, e / 2)), static_cast<float>(ldexp(1.0, e - e / 2)));
}

// X_0, scaled, as planes [2][B][M][pitch]; with DIRECT (no steps) scale * X_0 to y.
template <bool DIRECT>
__global__ void __launch_bounds__(256) start_kernel(const char *x, int type, int64_t nb_row, int64_t nb_mat, int64_t N, int64_t M,
                                                    bool wide, const double *sums, int parts, float eps, __half *dst, int64_t pitch,
                                                    char *y, int y_type, int64_t nb_y, int64_t nb_y_mat, float scale) {
    __shared__ float2 factors;
    if (threadIdx.x < 32) {
        const float2 f = inverse_norm(sums + static_cast<int64_t>(blockIdx.y) * parts, parts, eps);
        if (threadIdx.x == 0) factors = f;
    }
    __syncthreads();
    const float2 f = factors;
    const char *p = x + blockIdx.y * nb_mat;
    const int64_t plane = gridDim.y * M * pitch, spans = (N + kSpan - 1) / kSpan;
    for (int64_t i = blockIdx.x * 8LL + (threadIdx.x >> 5); i < M * spans; i += gridDim.x * 8LL) {
        const int64_t r = i / spans, c0 = (i - r * spans) * kSpan, end = min(N, c0 + kSpan);
#pragma unroll 4
        for (int64_t c = c0 + (threadIdx.x & 31) * 8; c < end; c += 256) {
            float v[8];
            load8(p + r * nb_row, type, c, N, wide, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = v[k] * f.x * f.y;
            if constexpr (DIRECT) {
                char *row = y + blockIdx.y * nb_y_mat + r * nb_y;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (c + k >= N) continue;
                    if (y_type == OOP_TYPE_F32) reinterpret_cast<float *>(row)[c + k] = scale * v[k];
                    else reinterpret_cast<__nv_bfloat16 *>(row)[c + k] = __float2bfloat16_rn(scale * v[k]);
                }
            } else {                                       // whole pitches
                __half hi[8], lo[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    hi[k] = __float2half_rn(v[k] * kScaleX);
                    lo[k] = __float2half_rn(v[k] * kScaleX - __half2float(hi[k]));
                }
                __half *d = dst + (blockIdx.y * M + r) * pitch + c;
                uint4 w;
                __builtin_memcpy(&w, hi, 16);
                *reinterpret_cast<uint4 *>(d) = w;
                __builtin_memcpy(&w, lo, 16);
                *reinterpret_cast<uint4 *>(d + plane) = w;
            }
        }
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

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }

size_t plane_pair_bytes(int64_t cols, int64_t rows, int64_t B) {
    return round256(static_cast<size_t>(2 * B * rows * round8(cols)) * 2);
}

// B matrices of two planes: [2][B][rows][pitch].
struct Planes {
    char *p;
    int64_t cols, rows, B;
    int64_t pitch() const { return round8(cols); }
    int64_t matrix_bytes() const { return rows * pitch() * 2; }
    __half *hi() const { return reinterpret_cast<__half *>(p); }
    __half *lo() const { return reinterpret_cast<__half *>(p + B * matrix_bytes()); }
    pair::Operand operand(bool rows_contiguous) const {
        return {p, cols, rows, pitch() * 2, matrix_bytes(), 2 * B, rows_contiguous, true};
    }
};

// A product of two such operands over all matrices.
pair::Spec product_of(const Planes &a, bool a_rows, const Planes &b, bool b_rows, int64_t M, int64_t N, int64_t K) {
    pair::Spec s = {};
    s.a = a.operand(a_rows);
    s.b[0] = s.b[1] = b.operand(b_rows);
    s.M = M, s.N = N, s.K = K;
    s.batches = static_cast<int>(a.B);
    s.segments = 1;
    s.planes_a = s.planes_b = 2;
    s.a_plane = s.b_plane = static_cast<int>(a.B);
    s.a_batch = s.b_batch = 1;
    return s;
}

void to_planes(pair::Spec &s, const Planes &d, float alpha) {
    s.out.p0 = d.hi();
    s.out.p1 = d.lo();
    s.out.nb0 = d.pitch() * 2;
    s.out.batch = d.matrix_bytes();
    s.out.alpha = alpha;
}

}  // namespace
}  // namespace oop

using namespace oop;

extern "C" {

size_t oop_orthogonalise_workspace_size(const int64_t ne[3]) {
    if (check_sizes(ne) != OOP_OK || ne[0] == 0 || ne[1] == 0 || ne[2] == 0) return 0;
    const int64_t n = std::min(ne[0], ne[1]);
    return round256(static_cast<size_t>(ne[2] * parts_of(ne[0] * ne[1])) * sizeof(double)) +
           2 * plane_pair_bytes(ne[0], ne[1], ne[2]) + 2 * plane_pair_bytes(n, n, ne[2]);
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
    const int64_t n = std::min(M, N), deep = std::max(M, N);
    const bool tall = M > N;
    const int parts = static_cast<int>(parts_of(M * N));
    double *sums = static_cast<double *>(workspace);
    char *at = static_cast<char *>(workspace) + round256(static_cast<size_t>(B * parts) * sizeof(double));
    Planes X = {at, N, M, B}, next = {at + plane_pair_bytes(N, M, B), N, M, B};
    const Planes A = {next.p + plane_pair_bytes(N, M, B), n, n, B}, Q = {A.p + plane_pair_bytes(n, n, B), n, n, B};
    const char *xp = static_cast<const char *>(x);
    char *yp = static_cast<char *>(y);
    const unsigned nb = static_cast<unsigned>(B);
    const bool wide = is_aligned(x, 16) && (M <= 1 || nb_x[0] % 16 == 0) && (B <= 1 || nb_x[1] % 16 == 0);
    const int64_t units = M * ((N + kSpan - 1) / kSpan);
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((units + 7) / 8, 1216));
    squares_kernel<<<dim3(static_cast<unsigned>(parts), nb), 256, 0, st>>>(xp, x_type, nb_x[0], nb_x[1], N, M, wide, sums);
    if (steps == 0)
        start_kernel<true><<<dim3(blocks, nb), 256, 0, st>>>(xp, x_type, nb_x[0], nb_x[1], N, M, wide, sums, parts, eps, nullptr, 0, yp,
                                                             y_type, nb_y[0], nb_y[1], scale);
    else
        start_kernel<false><<<dim3(blocks, nb), 256, 0, st>>>(xp, x_type, nb_x[0], nb_x[1], N, M, wide, sums, parts, eps, X.hi(), X.pitch(),
                                                              nullptr, 0, 0, 0, 0.f);
    g_kernel_launches = 2;
    cudaError_t e = cudaGetLastError();
    for (int i = 0; i < steps && e == cudaSuccess; ++i) {
        const float *c = coefs ? coefs + 3 * i : kDefault;
        pair::Spec s = product_of(X, tall, X, tall, n, n, deep);               // A = X X', or X' X
        s.symmetric = true;
        to_planes(s, A, kScaleA / (kScaleX * kScaleX));
        e = pair::launch<pair::kSplit, true, 256>(s, status, st);
        if (e != cudaSuccess) break;
        s = product_of(A, false, A, false, n, n, n);                           // Q = a + b A + c A A
        s.symmetric = s.a_half = s.b_half = true;
        to_planes(s, Q, c[2] * (kScaleQ / (kScaleA * kScaleA)));
        s.out.c_hi = A.hi();
        s.out.c_lo = A.lo();
        s.out.beta = c[1] * (kScaleQ / kScaleA);
        s.out.diag = c[0] * kScaleQ;
        e = pair::launch<pair::kSplit, true, 256>(s, status, st);
        if (e != cudaSuccess) break;
        s = tall ? product_of(X, false, Q, false, M, N, N) : product_of(Q, false, X, true, M, N, M);   // X Q, or Q X
        s.a_half = !tall;
        s.b_half = tall;
        if (i + 1 < steps) {
            to_planes(s, next, 1.f / kScaleQ);
            e = pair::launch<pair::kSplit, true, 256>(s, status, st);
        } else {
            s.out.p0 = yp;
            s.out.nb0 = nb_y[0];
            s.out.batch = nb_y[1];
            s.out.type = y_type;
            s.out.alpha = scale / (kScaleQ * kScaleX);
            s.out.wide = N * ys % 16 == 0 && is_aligned(y, 16) && (M <= 1 || nb_y[0] % 16 == 0) && (B <= 1 || nb_y[1] % 16 == 0);
            e = pair::launch<pair::kPlain, true, 256>(s, status, st);
        }
        std::swap(X, next);
    }
    return cuda_status(e);
}

}  // extern "C"
