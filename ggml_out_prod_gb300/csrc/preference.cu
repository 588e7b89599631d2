// preference.cu -- a preference loss over pairs of sequences, from logits, and
// its gradient.
//
//   lse[t]   = log sum_v exp(x[v, t]),  logp[t] = x[label[t], t] - lse[t]
//   ratio[s] = sum over the scored rows t of sequence s of logp[t] - ref[t]
//   m_i      = beta * (ratio[i] - ratio[P + i])           chosen, rejected
//   loss_i   = -(1 - e) log sigma(m_i) - e log sigma(-m_i),  loss = mean_i loss_i
//
//   dx[v, t] = c_s * (1[v = label[t]] - exp(x[v, t] - lse[t])),
//   c_i = -c_{P+i} = dloss * beta / P * (e sigma(m_i) - (1 - e) sigma(-m_i))
//
// A row whose label is negative is not scored: its logits are not read.
//
// The paired ratios are sums of small per-token differences, taken in 64 bits:
// the difference of two sums of log probabilities would cancel.
#include <algorithm>
#include <cmath>

#include "oop_internal.cuh"
#include "rows.cuh"

namespace oop {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kChunk = 16384;    // elements of a row that one CTA sums
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// sum_i exp(x_i) = s * exp(m), m the largest x (or -Inf and s = 0: no terms).
struct LogSum {
    float m, s;
};

__device__ __forceinline__ LogSum join(LogSum a, LogSum b) {
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY) return {m, a.s + b.s};
    // equal maxima (infinite ones too) scale by one
    const float fa = a.m == m ? 1.f : exp2_fast((a.m - m) * kLog2e);
    const float fb = b.m == m ? 1.f : exp2_fast((b.m - m) * kLog2e);
    return {m, a.s * fa + b.s * fb};
}

// One term; a NaN stays in s, where no maximum can lose it.
__device__ __forceinline__ LogSum term(float x) {
    return isnan(x) ? LogSum{-INFINITY, x} : LogSum{x, 1.f};
}

// log(s) in 64 bits: the log of the sum is m + log(s).
__device__ __forceinline__ double log_of(LogSum r) {
    return r.m == -INFINITY && !isnan(r.s) ? 0.0 : log(static_cast<double>(r.s));
}

struct Workspace {
    double *ratio;       // {2P}
    int *done;           // sequences finished
    LogSum *part;        // {chunks, T}
};

Workspace carve(void *ws, int64_t pairs) {
    char *p = static_cast<char *>(ws);
    Workspace w;
    w.done = reinterpret_cast<int *>(p);
    w.ratio = reinterpret_cast<double *>(p + 256);
    w.part = reinterpret_cast<LogSum *>(p + 256 + (2 * pairs * 8 + 255) / 256 * 256);
    return w;
}

int64_t chunks_of(int64_t V) { return std::max<int64_t>(1, (V + kChunk - 1) / kChunk); }

struct LossArgs {
    const void *x;
    const int32_t *labels, *seq;
    const float *ref;
    float *loss, *losses, *ratios, *logps, *lse;
    int64_t nb_x, V, T, P, chunks;
    double beta, smoothing;
    Workspace ws;
    int *status;
};

template <int XT>
__global__ void __launch_bounds__(kThreads) loss_part_kernel(const LossArgs a) {
    __shared__ LogSum part[kThreads / 32];
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ws.done = 0;
    const int64_t t = blockIdx.x / a.chunks, c = blockIdx.x - t * a.chunks;
    const int32_t label = a.labels[t];
    if (label < 0 || label >= a.V) return;
    const auto *x = row_of<XT>(a.x, a.nb_x, t);
    const int64_t v1 = min(a.V, (c + 1) * kChunk);
    LogSum r = {-INFINITY, 0.f};
    for (int64_t v = c * kChunk + threadIdx.x; v < v1; v += kThreads)
        r = join(r, term(to_float(x[v])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        r = join(r, LogSum{__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o)});
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = r;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) r = join(r, part[w]);
        a.ws.part[t * a.chunks + c] = r;
    }
}

__device__ __forceinline__ double softplus(double x) {      // log(1 + exp(x))
    return fmax(x, 0.0) + log1p(exp(-fabs(x)));
}

// One CTA per sequence joins its rows' partial sums; the last CTA to finish
// takes the pairs.  Without pairs, one CTA per kThreads rows.
template <int XT>
__global__ void __launch_bounds__(kThreads) loss_join_kernel(const LossArgs a) {
    __shared__ double part[32];
    __shared__ bool last;
    const int64_t n_seq = 2 * a.P, s = blockIdx.x;
    int64_t t0 = 0, t1 = 0;            // the rows written here
    int64_t s0 = 0, s1 = 0;            // those of them in the sequence
    if (a.P == 0) {
        t0 = s * kThreads;
        t1 = min(a.T, t0 + kThreads);
    } else {
        const int64_t b0 = a.seq[s], b1 = a.seq[s + 1];
        if (threadIdx.x == 0 && (b0 < 0 || b1 < b0 || b1 > a.T)) record_status(a.status, OOP_ERR_BAD_ID);
        s0 = min(max(b0, int64_t(0)), a.T);
        s1 = min(max(b1, s0), a.T);
        t0 = s == 0 ? 0 : s0;
        t1 = s == n_seq - 1 ? a.T : s1;
    }
    double sum = 0.0;
    for (int64_t t = t0 + threadIdx.x; t < t1; t += kThreads) {
        const int32_t label = a.labels[t];
        float lse = 0.f, logp = 0.f;
        if (label >= a.V) record_status(a.status, OOP_ERR_BAD_ID);
        if (label >= 0 && label < a.V) {
            LogSum r = a.ws.part[t * a.chunks];
            for (int64_t c = 1; c < a.chunks; ++c) r = join(r, a.ws.part[t * a.chunks + c]);
            const double z = log_of(r), top = r.m;
            // x - top first: it is exact, where top + log(s) may lose log(s)
            const double lp = (static_cast<double>(to_float(row_of<XT>(a.x, a.nb_x, t)[label])) - top) - z;
            lse = static_cast<float>(top + z);
            logp = static_cast<float>(lp);
            if (t >= s0 && t < s1) sum += lp - (a.ref ? static_cast<double>(a.ref[t]) : 0.0);
        }
        a.lse[t] = lse;
        a.logps[t] = logp;
    }
    if (a.P == 0) return;
    sum = block_sum(sum, part);
    if (threadIdx.x == 0) {
        a.ws.ratio[s] = sum;
        a.ratios[s] = static_cast<float>(sum);
        __threadfence();
        last = atomicAdd(a.ws.done, 1) == n_seq - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    sum = 0.0;
    for (int64_t i = threadIdx.x; i < a.P; i += kThreads) {
        const double m = a.beta * (__ldcg(a.ws.ratio + i) - __ldcg(a.ws.ratio + a.P + i));
        const double e = a.smoothing;
        const double l = (1.0 - e) * softplus(-m) + (e > 0.0 ? e * softplus(m) : 0.0);
        a.losses[i] = static_cast<float>(l);
        sum += l;
    }
    sum = block_sum(sum, part);
    if (threadIdx.x == 0) *a.loss = static_cast<float>(sum / static_cast<double>(a.P));
}

struct LossBackArgs {
    const void *x;
    const int32_t *labels, *seq;
    const float *lse, *ratios, *dloss;
    void *dx;
    int64_t nb_x, nb_dx, V, T, P, chunks;
    double beta, smoothing;
    int *status;
};

// d(loss) / d(logp) of a row of sequence s.
__device__ __forceinline__ float slope_of(const LossBackArgs &a, int64_t s) {
    const int64_t i = s < a.P ? s : s - a.P;
    const double m = a.beta * (static_cast<double>(a.ratios[i]) - a.ratios[a.P + i]);
    const double e = a.smoothing;
    const double up = a.dloss ? static_cast<double>(*a.dloss) : 1.0;
    const double c = up * a.beta / static_cast<double>(a.P) *
                     (e / (1.0 + exp(-m)) - (1.0 - e) / (1.0 + exp(m)));
    return static_cast<float>(s < a.P ? c : -c);
}

// The sequence that holds row t, or -1: the last s with seq[s] <= t.
__device__ __forceinline__ int64_t sequence_of(const LossBackArgs &a, int64_t t) {
    int64_t lo = 0, hi = 2 * a.P + 1;             // seq[lo - 1] <= t < seq[hi]
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (a.seq[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    return lo - 1 < 2 * a.P ? lo - 1 : -1;
}

template <int XT, int DT>
__global__ void __launch_bounds__(kThreads) loss_back_kernel(const LossBackArgs a) {
    __shared__ float coef;
    const int64_t t = blockIdx.x / a.chunks, c = blockIdx.x - t * a.chunks;
    const int64_t v0 = c * kChunk, v1 = min(a.V, v0 + kChunk);
    const int32_t label = a.labels[t];
    auto *dx = row_of<DT>(a.dx, a.nb_dx, t);
    if (threadIdx.x == 0) {
        if (label >= a.V) record_status(a.status, OOP_ERR_BAD_ID);
        const int64_t s = label >= 0 && label < a.V && a.P > 0 ? sequence_of(a, t) : -1;
        coef = s >= 0 ? slope_of(a, s) : 0.f;
    }
    __syncthreads();
    const float k = coef;
    if (label < 0 || label >= a.V || k == 0.f) {
        for (int64_t v = v0 + threadIdx.x; v < v1; v += kThreads) dx[v] = from_float<DT>(0.f);
        return;
    }
    const auto *x = row_of<XT>(a.x, a.nb_x, t);
    const float lse = a.lse[t];
    for (int64_t v = v0 + threadIdx.x; v < v1; v += kThreads) {
        const float p = exp2_fast((to_float(x[v]) - lse) * kLog2e);
        dx[v] = from_float<DT>(k * ((v == label ? 1.f : 0.f) - p));
    }
}

int check_loss(const int64_t ne[2], int64_t pairs) {
    if (!ne) return OOP_ERR_NULL;
    const int rc = check_extent(ne[0], ne[1]);
    if (rc != OOP_OK) return rc;
    if (pairs < 0 || pairs > 0x3fffffffLL || ne[0] > 0x7fffffffLL || ne[1] > 0x7fffffffLL)
        return OOP_ERR_SHAPE;
    if (chunks_of(ne[0]) * ne[1] > 0x7fffffffLL) return OOP_ERR_SHAPE;   // CTAs ride grid.x
    return OOP_OK;
}

int check_scalars(double beta, double smoothing) {
    return std::isfinite(beta) && smoothing >= 0.0 && smoothing <= 1.0 ? OOP_OK : OOP_ERR_VALUE;
}

template <int XT>
void launch_loss(const LossArgs &a, cudaStream_t st) {
    if (a.T > 0) loss_part_kernel<XT><<<static_cast<unsigned>(a.T * a.chunks), kThreads, 0, st>>>(a);
    const int64_t grid = a.P > 0 ? 2 * a.P : (a.T + kThreads - 1) / kThreads;
    if (grid > 0) loss_join_kernel<XT><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a);
}

}  // namespace
}  // namespace oop

using namespace oop;

extern "C" {

size_t oop_preference_loss_workspace_size(const int64_t ne[2], int64_t n_pairs) {
    if (check_loss(ne, n_pairs) != OOP_OK) return 0;
    return 256 + static_cast<size_t>(2 * n_pairs * 8 + 255) / 256 * 256 +
           static_cast<size_t>(ne[1] * chunks_of(ne[0])) * sizeof(LogSum);
}

int oop_preference_loss(const void *logits, int type, int64_t nb, const int32_t *labels,
                        const int32_t *seq, const float *ref_logps, float *loss, float *losses,
                        float *ratios, float *logps, float *lse, const int64_t ne[2],
                        int64_t n_pairs, double beta, double label_smoothing, void *workspace,
                        size_t workspace_bytes, void *stream) {
    g_kernel_launches = 0;
    int rc = check_loss(ne, n_pairs);
    if (rc != OOP_OK) return rc;
    const int64_t V = ne[0], T = ne[1];
    const int size = plain_size(type);
    if (!size) return OOP_ERR_TYPE;
    if ((rc = check_scalars(beta, label_smoothing)) != OOP_OK) return rc;
    if ((rc = check_row_stride(V * size, T, nb, size, false)) != OOP_OK) return rc;
    if (T > 0) {
        if (V > 0 && (rc = check_pointer(logits, size)) != OOP_OK) return rc;
        if ((rc = check_pointer(labels, 4)) != OOP_OK) return rc;
        if ((rc = check_pointer(logps, 4)) != OOP_OK) return rc;
        if ((rc = check_pointer(lse, 4)) != OOP_OK) return rc;
        if (!is_aligned(ref_logps, 4)) return OOP_ERR_ALIGN;
    }
    if (n_pairs > 0) {
        if ((rc = check_pointer(seq, 4)) != OOP_OK) return rc;
        if ((rc = check_pointer(losses, 4)) != OOP_OK) return rc;
        if ((rc = check_pointer(ratios, 4)) != OOP_OK) return rc;
        if ((rc = check_pointer(loss, 4)) != OOP_OK) return rc;
    }
    if (T == 0 && n_pairs == 0) return OOP_OK;
    if (!workspace || workspace_bytes < oop_preference_loss_workspace_size(ne, n_pairs) ||
        !is_aligned(workspace, 256))
        return OOP_ERR_WORKSPACE;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const LossArgs a = {logits, labels, seq, ref_logps, loss, losses, ratios, logps, lse, nb, V, T,
                        n_pairs, chunks_of(V), beta, label_smoothing, carve(workspace, n_pairs),
                        status};
    cudaError_t e = cudaSuccess;
    if (T == 0) e = cudaMemsetAsync(a.ws.done, 0, sizeof(int), st);
    if (e != cudaSuccess) return cuda_status(e);
    if (type == OOP_TYPE_F32) launch_loss<OOP_TYPE_F32>(a, st);
    else if (type == OOP_TYPE_F16) launch_loss<OOP_TYPE_F16>(a, st);
    else launch_loss<OOP_TYPE_BF16>(a, st);
    e = cudaGetLastError();
    if (e == cudaSuccess) g_kernel_launches = T > 0 ? 2 : 1;
    return cuda_status(e);
}

int oop_preference_loss_back(const void *logits, int type, int64_t nb, const int32_t *labels,
                             const int32_t *seq, const float *lse, const float *ratios,
                             const float *dloss, void *dlogits, int d_type, int64_t nb_d,
                             const int64_t ne[2], int64_t n_pairs, double beta,
                             double label_smoothing, void *stream) {
    g_kernel_launches = 0;
    int rc = check_loss(ne, n_pairs);
    if (rc != OOP_OK) return rc;
    const int64_t V = ne[0], T = ne[1];
    const int size = plain_size(type), dsize = plain_size(d_type);
    if (!size || !gradient_type(d_type)) return OOP_ERR_TYPE;
    if ((rc = check_scalars(beta, label_smoothing)) != OOP_OK) return rc;
    if ((rc = check_row_stride(V * size, T, nb, size, false)) != OOP_OK) return rc;
    if ((rc = check_row_stride(V * dsize, T, nb_d, dsize, true)) != OOP_OK) return rc;
    if (T == 0 || V == 0) return OOP_OK;
    if ((rc = check_pointer(logits, size)) != OOP_OK) return rc;
    if ((rc = check_pointer(labels, 4)) != OOP_OK) return rc;
    if ((rc = check_pointer(lse, 4)) != OOP_OK) return rc;
    if ((rc = check_pointer(dlogits, dsize)) != OOP_OK) return rc;
    if (n_pairs > 0) {
        if ((rc = check_pointer(seq, 4)) != OOP_OK) return rc;
        if ((rc = check_pointer(ratios, 4)) != OOP_OK) return rc;
    }
    if (!is_aligned(dloss, 4)) return OOP_ERR_ALIGN;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const LossBackArgs a = {logits, labels, seq, lse, ratios, dloss, dlogits, nb, nb_d, V, T,
                            n_pairs, chunks_of(V), beta, label_smoothing, status};
    void (*kern)(LossBackArgs) = nullptr;
    const bool f32 = d_type == OOP_TYPE_F32;
    switch (type) {
    case OOP_TYPE_F32:
        kern = f32 ? loss_back_kernel<OOP_TYPE_F32, OOP_TYPE_F32> : loss_back_kernel<OOP_TYPE_F32, OOP_TYPE_BF16>;
        break;
    case OOP_TYPE_F16:
        kern = f32 ? loss_back_kernel<OOP_TYPE_F16, OOP_TYPE_F32> : loss_back_kernel<OOP_TYPE_F16, OOP_TYPE_BF16>;
        break;
    default:
        kern = f32 ? loss_back_kernel<OOP_TYPE_BF16, OOP_TYPE_F32> : loss_back_kernel<OOP_TYPE_BF16, OOP_TYPE_BF16>;
    }
    kern<<<static_cast<unsigned>(T * a.chunks), kThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) g_kernel_launches = 1;
    return cuda_status(e);
}

}  // extern "C"
