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
#include <algorithm>
#include <cmath>

#include "oop_internal.cuh"
#include "rows.cuh"

namespace oop {
namespace {

constexpr int kThreads = 256;
// Fewer rows than this: as many threads per row as it has vectors, for latency.
constexpr int64_t kFewRows = 2048;
constexpr int64_t kSlices = 152;     // row slices of the weight's gradient: one per SM

struct NormArgs {
    const void *x, *w, *b;
    void *y;
    float *mean, *rstd;
    int64_t nb_x, nb_y, M, T;
    int w_type, width;
    float eps;
};

// Column m0 .. m0 + E - 1 of a parameter of a run-time type (E = 1, or 16-byte
// aligned rows and m0 % E == 0).
template <int E>
__device__ __forceinline__ void load_params(const void *p, int type, int64_t m0, float (&v)[E]) {
    if (type == OOP_TYPE_F32) {
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

// The sum over the `width` threads (a power of two, 32 or more) that share a
// row; every thread of the CTA calls it.
__device__ __forceinline__ float row_sum(float v, int width, float *part) {
    v = warp_sum(v);
    if (width == 32) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = width >> 5;
    __syncthreads();          // part may still be read by an earlier call
    if (lane == 0) part[warp] = v;
    __syncthreads();
    return warp_sum(lane < warps ? part[(warp & ~(warps - 1)) + lane] : 0.f);
}

// `width` threads per row hold it whole: NV vectors of E elements each, every
// load before the first use, so the mean, the squares and the result read
// registers.
template <int XT, int YT, int E, int NV>
__global__ void __launch_bounds__(1024) norm_kernel(const NormArgs a) {
    __shared__ float part[32];
    const int lane = static_cast<int>(threadIdx.x) & (a.width - 1);
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / a.width) + threadIdx.x / a.width;
    const bool in = t < a.T;
    const int M = static_cast<int>(a.M), step = a.width * E;
    const auto *x = row_of<XT>(a.x, a.nb_x, in ? t : 0);
    Packed<XT, E> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (in && i * step + lane * E < M) raw[i] = load_stream<XT, E>(x + i * step + lane * E);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (i * step + lane * E >= M) continue;
        float v[E];
        raw[i].get(v);
#pragma unroll
        for (int e = 0; e < E; ++e) s += v[e];
    }
    const float mean = row_sum(s, a.width, part) / static_cast<float>(M);
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (i * step + lane * E >= M) continue;
        float v[E];
        raw[i].get(v);
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(v[e] - mean, v[e] - mean, s);
    }
    const float rstd = 1.f / sqrtf(row_sum(s, a.width, part) / static_cast<float>(M) + a.eps);
    if (!in) return;
    auto *y = row_of<YT>(a.y, a.nb_y, t);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int m = i * step + lane * E;
        if (m >= M) continue;
        float v[E], p[E];
        raw[i].get(v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = (v[e] - mean) * rstd;
        if (a.w) {
            load_params<E>(a.w, a.w_type, m, p);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] *= p[e];
        }
        if (a.b) {
            load_params<E>(a.b, a.w_type, m, p);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] += p[e];
        }
        store_stream<YT, E>(y + m, v);
    }
    if (lane == 0) {
        if (a.mean) a.mean[t] = mean;
        if (a.rstd) a.rstd[t] = rstd;
    }
}

// Rows that 1024 threads cannot hold: one CTA per row, read three times (the
// second and third time from L2).
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

constexpr int kBackCols = 16;        // columns of one thread
constexpr int kMaxStages = 4;

// dx, and this CTA's part of dw and db, in one pass.  `width` threads share a
// row, 16 columns each, and keep the columns' sums in registers over all the
// rows they meet; a CTA (one per SM) has `groups` such rows in work, and each
// thread copies its pieces of the next rows into shared memory while this one
// is reduced, so the loads never wait for the row's two sums.
template <int XT, int DT, int E, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) norm_back_kernel(const NormBackArgs a) {
    constexpr int NV = kBackCols / E;
    constexpr int BX = E * plain_size(XT), BD = E * plain_size(DT);
    constexpr bool kAsync = BX >= 4 && BD >= 4;      // 2-byte pieces are loaded when they are due
    extern __shared__ __align__(16) char sm[];
    let_next_start();
    const int M = static_cast<int>(a.M), threads = blockDim.x, tid = threadIdx.x;
    float *ws = reinterpret_cast<float *>(sm);                       // w as floats
    float2 *red = reinterpret_cast<float2 *>(sm + ((M + 3) & ~3) * 4);   // {2, 32}
    char *ring = reinterpret_cast<char *>(red + 64);
    const int stage_bytes = threads * NV * (BX + BD);
    for (int m = tid; m < M; m += threads) ws[m] = a.w ? load_any(a.w, a.w_type, m) : 1.f;
    __syncthreads();

    const int group = tid / a.width, lane = tid - group * a.width;
    const int warps = a.width >> 5, warp0 = group * warps;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * a.groups + group;
    const int64_t step = static_cast<int64_t>(gridDim.x) * a.groups;
    auto slot_x = [&](int st, int i) { return ring + st * stage_bytes + (i * threads + tid) * BX; };
    auto slot_d = [&](int st, int i) {
        return ring + st * stage_bytes + threads * NV * BX + (i * threads + tid) * BD;
    };
    auto issue = [&](int64_t t, int st) {
        if (kAsync && t < a.T) {
            const auto *x = row_of<XT>(a.x, a.nb_x, t);
            const auto *d = row_of<DT>(a.dy, a.nb_dy, t);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int m = (i * a.width + lane) * E;
                if (m < M) {
                    if constexpr (kAsync) {
                        copy_async<BX>(slot_x(st, i), x + m);
                        copy_async<BD>(slot_d(st, i), d + m);
                    }
                }
            }
        }
        if (kAsync) commit_copies();
    };
    float dw[NV][E], db[NV][E];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) dw[i][e] = db[i][e] = 0.f;

    for (int s = 0; s + 1 < a.stages; ++s) issue(r0 + s * step, s);
    float mean_next = 0.f, rstd_next = 0.f;
    if (r0 < a.T) {
        mean_next = a.mean[r0];
        rstd_next = a.rstd[r0];
    }
    int st = 0, odd = 0;
    for (int64_t t = r0; t < a.T; t += step) {
        const int fill = st == 0 ? a.stages - 1 : st - 1;
        issue(t + (a.stages - 1) * step, fill);
        const float mean = mean_next, rstd = rstd_next;
        if (t + step < a.T) {
            mean_next = a.mean[t + step];
            rstd_next = a.rstd[t + step];
        }
        if (kAsync) wait_copies(a.stages - 1);
        Packed<XT, E> xr[NV];
        Packed<DT, E> dr[NV];
        float2 sum = make_float2(0.f, 0.f);
        const auto *x = row_of<XT>(a.x, a.nb_x, t);
        const auto *d = row_of<DT>(a.dy, a.nb_dy, t);
        if constexpr (!kAsync) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int m = (i * a.width + lane) * E;
                if (m < M) {
                    xr[i] = load_stream<XT, E>(x + m);
                    dr[i] = load_stream<DT, E>(d + m);
                }
            }
        }
        auto columns = [&](int i, float (&xh)[E], float (&g)[E], float (&dv)[E], int m) {
            if constexpr (kAsync) {
                xr[i].raw = *reinterpret_cast<const decltype(xr[i].raw) *>(slot_x(st, i));
                dr[i].raw = *reinterpret_cast<const decltype(dr[i].raw) *>(slot_d(st, i));
            }
            float w[E];
            load_params<E>(ws, OOP_TYPE_F32, m, w);
            xr[i].get(xh);
            dr[i].get(dv);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                xh[e] = (xh[e] - mean) * rstd;
                g[e] = dv[e] * w[e];
            }
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int m = (i * a.width + lane) * E;
            if (m >= M) continue;
            float xh[E], g[E], dv[E];
            columns(i, xh, g, dv, m);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                sum.x += g[e];
                sum.y = fmaf(g[e], xh[e], sum.y);
                dw[i][e] = fmaf(dv[e], xh[e], dw[i][e]);
                db[i][e] += dv[e];
            }
        }
        sum.x = warp_sum(sum.x);
        sum.y = warp_sum(sum.y);
        if (warps > 1) {
            float2 *now = red + odd * 32;            // the other half may still be read
            if ((tid & 31) == 0) now[tid >> 5] = sum;
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(a.width) : "memory");
            sum = (tid & 31) < warps ? now[warp0 + (tid & 31)] : make_float2(0.f, 0.f);
            sum.x = warp_sum(sum.x);
            sum.y = warp_sum(sum.y);
            odd ^= 1;
        }
        const float mg = sum.x / static_cast<float>(M), mgx = sum.y / static_cast<float>(M);
        auto *dx = row_of<DT>(a.dx, a.nb_dx, t);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int m = (i * a.width + lane) * E;
            if (m >= M) continue;
            float xh[E], g[E], dv[E];
            columns(i, xh, g, dv, m);
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] = rstd * (g[e] - mg - xh[e] * mgx);
            store_stream<DT, E>(dx + m, g);
        }
        st = st + 1 == a.stages ? 0 : st + 1;
    }
    if (!a.part) return;
    // the groups' sums, group after group
    if (kAsync) wait_copies(0);
    float *all = reinterpret_cast<float *>(ring);
    for (int k = 0; k < a.groups; ++k) {
        if (a.groups > 1) __syncthreads();
        if (group != k) continue;
        const bool first = k == 0, last = k == a.groups - 1;
        float *out = a.part + static_cast<int64_t>(blockIdx.x) * M;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int m = (i * a.width + lane) * E;
            if (m >= M) continue;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float sw = first ? dw[i][e] : all[m + e] + dw[i][e];
                const float sb = first ? db[i][e] : all[M + m + e] + db[i][e];
                (last ? out : all)[m + e] = sw;
                (last ? out + static_cast<int64_t>(gridDim.x) * M : all + M)[m + e] = sb;
            }
        }
    }
}

// Rows of more than 16384 columns: dx from one CTA per row, then the columns'
// sums.
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
    if (m < M) {
#pragma unroll 20
        for (int k = warp; k < slices; k += kThreads / 32) s += __ldcg(part + k * M);
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp > 0 || m >= M) return;
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) s += sums[w][lane];
    out[m] = s;
}

int64_t slices_of(int64_t T) { return T < kSlices ? T : kSlices; }

// Vectors a thread of the row kernel holds at most.
constexpr int kNormVecs = 8, kNormSingles = 16;

template <int XT, int YT>
void launch_norm(NormArgs a, bool wide, cudaStream_t st) {
    // 16 bytes of the narrower type, so that neither side moves less
    constexpr int E = plain_size(XT) == 2 && plain_size(YT) == 2 ? 8 : 4;
    const int64_t units = wide ? a.M / E : a.M;
    const int64_t most = wide ? kNormVecs : kNormSingles;
    if (units > 1024 * most) {
        norm_long_kernel<XT, YT><<<static_cast<unsigned>(a.T), kThreads, 0, st>>>(a);
        return;
    }
    a.width = 32;
    while (a.width < 1024 && (units > a.width * most || (a.T < kFewRows && units > a.width))) a.width *= 2;
    const int threads = std::max(a.width, 128);
    const unsigned grid = static_cast<unsigned>((a.T + threads / a.width - 1) / (threads / a.width));
    if (wide) norm_kernel<XT, YT, E, kNormVecs><<<grid, threads, 0, st>>>(a);
    else norm_kernel<XT, YT, 1, kNormSingles><<<grid, threads, 0, st>>>(a);
}

template <int XT>
void launch_norm(const NormArgs &a, int yt, bool wide, cudaStream_t st) {
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

template <int XT, int DT, int E>
cudaError_t launch_back_kernel(NormBackArgs a, cudaStream_t st) {
    constexpr int bytes = kBackCols * (plain_size(XT) + plain_size(DT));
    constexpr bool async = E * plain_size(XT) >= 4 && E * plain_size(DT) >= 4;
    constexpr int most = async ? 1024 : 512;     // threads of a CTA
    a.width = static_cast<int>((a.M + 32 * kBackCols - 1) / (32 * kBackCols)) * 32;
    const int fixed = static_cast<int>((a.M + 3) / 4 * 16) + 64 * 8;
    const int slots = (220 * 1024 - fixed) / (a.width * bytes);      // rows that fit on chip
    // as many rows at once as fit, twice if they can be (one in work, one on its
    // way), but no CTA with many rows while others have none; named barriers
    // 1 .. 15 are theirs (a warp that has a row alone needs none)
    a.groups = static_cast<int>(std::min<int64_t>({most / a.width, a.width == 32 ? 16 : 15,
                                                   std::max(1, slots / 2), (a.T + kSlices - 1) / kSlices}));
    const int threads = a.width * a.groups;
    const int slices = static_cast<int>(std::min(kSlices, (a.T + a.groups - 1) / a.groups));
    a.stages = std::max(1, std::min(kMaxStages, slots / a.groups));
    const int ring = std::max(a.stages * threads * bytes, a.groups > 1 ? static_cast<int>(a.M) * 8 : 0);
    const auto kern = norm_back_kernel<XT, DT, E, most>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, fixed + ring);
    if (e != cudaSuccess) return e;
    kern<<<slices, threads, fixed + ring, st>>>(a);
    if (!a.part) return cudaGetLastError();
    e = cudaGetLastError();
    return e != cudaSuccess ? e : join_slices<XT, DT>(a, slices, st);
}

template <int XT, int DT>
cudaError_t launch_back(const NormBackArgs &a, bool wide, cudaStream_t st) {
    constexpr int E = plain_size(XT) == 2 && plain_size(DT) == 2 ? 8 : 4;
    const bool single = !wide && (plain_size(XT) == 2 || plain_size(DT) == 2);
    if (a.M <= (single ? 512 : 1024) * kBackCols) {
        g_kernel_launches = a.part ? 2 : 1;
        return wide ? launch_back_kernel<XT, DT, E>(a, st) : launch_back_kernel<XT, DT, 1>(a, st);
    }
    norm_back_row_kernel<XT, DT><<<static_cast<unsigned>(a.T), kThreads, 0, st>>>(a);
    g_kernel_launches = a.part ? 3 : 1;
    if (!a.part) return cudaGetLastError();
    const int64_t tiles = (a.M + kThreads - 1) / kThreads, slices = slices_of(a.T);
    norm_back_cols_kernel<XT, DT>
        <<<dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(slices)), kThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : join_slices<XT, DT>(a, static_cast<int>(slices), st);
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
    const NormArgs a = {x, w, b, y, mean, rstd, nb_x, nb_y, M, T, w_type, 0, eps};
    const bool wide = M % 8 == 0 && is_aligned(x, 16) && is_aligned(y, 16) && is_aligned(w, 16) &&
                      is_aligned(b, 16) && nb_x % 16 == 0 && nb_y % 16 == 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (x_type == OOP_TYPE_F32) launch_norm<OOP_TYPE_F32>(a, y_type, wide, st);
    else if (x_type == OOP_TYPE_F16) launch_norm<OOP_TYPE_F16>(a, y_type, wide, st);
    else launch_norm<OOP_TYPE_BF16>(a, y_type, wide, st);
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
                      nb_dy % 16 == 0 && nb_x % 16 == 0 && nb_dx % 16 == 0;
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
