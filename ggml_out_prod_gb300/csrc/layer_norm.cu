// layer_norm.cu -- layer norm over the rows of {M, T}, forward and backward.
//
//   y  = (x - mean) * rstd * w + b,   rstd = (var + eps)^(-1/2)
//   g  = dy * w,  xh = (x - mean) * rstd
//   dx = rstd * (g - mean(g) - xh * mean(g * xh))
//   dw = sum over rows of dy * xh,   db = sum over rows of dy
//
// var is the mean of (x - mean)^2, taken after the mean is known: the
// difference of the mean square and the squared mean cancels for rows far from
// zero.
#include <cmath>

#include "oop_internal.cuh"
#include "rows.cuh"

namespace oop {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kSlices = 152;     // row slices of the weight's gradient: one per SM

struct NormArgs {
    const void *x, *w, *b;
    void *y;
    float *mean, *rstd;
    int64_t nb_x, nb_y, M;
    int w_type;
    float eps;
};

template <int XT, int YT>
__global__ void __launch_bounds__(kThreads) norm_row_kernel(const NormArgs a) {
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
    float *dw, *db, *part;
    int64_t nb_dy, nb_x, nb_dx, M, T;
    int w_type;
};

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

__global__ void __launch_bounds__(kThreads) norm_back_join_kernel(const float *part, int64_t slices,
                                                                  int64_t M, float *dw, float *db) {
    const int64_t m = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (m >= M) return;
    float sw = 0.f, sb = 0.f;
    for (int64_t s = 0; s < slices; ++s) {
        sw += part[s * M + m];
        sb += part[(slices + s) * M + m];
    }
    if (dw) dw[m] = sw;
    if (db) db[m] = sb;
}

int64_t slices_of(int64_t T) { return T < kSlices ? T : kSlices; }

template <int XT>
void (*norm_kernel(int yt))(NormArgs) {
    switch (yt) {
    case OOP_TYPE_F32: return norm_row_kernel<XT, OOP_TYPE_F32>;
    case OOP_TYPE_F16: return norm_row_kernel<XT, OOP_TYPE_F16>;
    default: return norm_row_kernel<XT, OOP_TYPE_BF16>;
    }
}

template <int XT, int DT>
void launch_back(const NormBackArgs &a, bool cols, cudaStream_t st) {
    norm_back_row_kernel<XT, DT><<<static_cast<unsigned>(a.T), kThreads, 0, st>>>(a);
    if (!cols) return;
    const int64_t tiles = (a.M + kThreads - 1) / kThreads, slices = slices_of(a.T);
    norm_back_cols_kernel<XT, DT>
        <<<dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(slices)), kThreads, 0, st>>>(a);
    norm_back_join_kernel<<<static_cast<unsigned>(tiles), kThreads, 0, st>>>(a.part, slices, a.M,
                                                                            a.dw, a.db);
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
    const NormArgs a = {x, w, b, y, mean, rstd, nb_x, nb_y, M, w_type, eps};
    const auto kern = x_type == OOP_TYPE_F32   ? norm_kernel<OOP_TYPE_F32>(y_type)
                      : x_type == OOP_TYPE_F16 ? norm_kernel<OOP_TYPE_F16>(y_type)
                                               : norm_kernel<OOP_TYPE_BF16>(y_type);
    kern<<<static_cast<unsigned>(T), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
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
    const NormBackArgs a = {dy, x,     w,    mean,  rstd, dx, dw,
                            db, static_cast<float *>(workspace), nb_dy, nb_x, nb_dx, M, T, w_type};
    const bool f32 = dy_type == OOP_TYPE_F32;
    switch (x_type) {
    case OOP_TYPE_F32:
        f32 ? launch_back<OOP_TYPE_F32, OOP_TYPE_F32>(a, cols, st)
            : launch_back<OOP_TYPE_F32, OOP_TYPE_BF16>(a, cols, st);
        break;
    case OOP_TYPE_F16:
        f32 ? launch_back<OOP_TYPE_F16, OOP_TYPE_F32>(a, cols, st)
            : launch_back<OOP_TYPE_F16, OOP_TYPE_BF16>(a, cols, st);
        break;
    default:
        f32 ? launch_back<OOP_TYPE_BF16, OOP_TYPE_F32>(a, cols, st)
            : launch_back<OOP_TYPE_BF16, OOP_TYPE_BF16>(a, cols, st);
    }
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) g_kernel_launches = cols ? 3 : 1;
    return cuda_status(e);
}

}  // extern "C"
