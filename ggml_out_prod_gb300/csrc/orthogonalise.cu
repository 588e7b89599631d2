// orthogonalise.cu -- the update of a weight made nearly orthogonal by Newton-Schulz
// steps, as the Muon optimiser does it.
//
//   X_0 = x / (|x|_F + eps),  X <- a X + (b A + c A A) X,  A = X X'
//
// A is taken on the smaller side: with M > N, X <- X (a + b X'X + c (X'X)^2) is the same
// polynomial of the singular values.
//
// Bound by the tensor cores (three products of binary16 planes for one of 22 bits), whose
// sums are folded every 64 k, and for few rows by launches.  f32, five steps: 8 x 2560 13
// to 15 us, 32 x 768 x 2048 1.63 ms, 9728 x 2560 to bf16 1.28 ms (1.97 with the steps on X
// itself).
#include <algorithm>
#include <cmath>

#include "oop_internal.cuh"
#include "pair_product.cuh"
#include "rows.cuh"

namespace oop {
namespace {

constexpr int kMaxSteps = 64;
constexpr float kDefault[3] = {3.4445f, -4.7750f, 2.0315f};

// The matrices between the products are held as two binary16 planes, hi + lo, of a scaled
// value: 22 bits or more, as many as a product of three terms keeps.  The scales leave
// room for magnitudes of 8, 64 and 256 below binary16's largest, and keep the planes of a
// 4096 x 4096 matrix (X's elements are about 2^-12) out of its subnormals; an element below
// 2^-16 of X, 2^-13 of A or 2^-11 of Q is off by up to 2^-38, 2^-35 or 2^-33.  bfloat16 planes
// would need no scale, but three of them and six terms.
constexpr float kScaleX = 0x1p13f, kScaleA = 0x1p10f, kScaleQ = 0x1p8f;

// Sums of squares: those of large, ordinary and small magnitudes apart, scaled so that
// none over- or underflows (the idea of Blue, "A portable Fortran program to find the
// Euclidean norm of a vector", TOMS 1978).
constexpr float kBigScale = 0x1p-80f, kSmallScale = 0x1p90f;

struct Squares {
    float big = 0.f, mid = 0.f, small = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float m = fabsf(v);
        if (m > 0x1p50f) {
            const float s = v * kBigScale;
            big = fmaf(s, s, big);
        } else if (m < 0x1p-40f) {
            const float s = v * kSmallScale;
            small = fmaf(s, s, small);
        } else {
            mid = fmaf(v, v, mid);                         // and NaN
        }
    }
};

// 1 / (|x|_F + eps) as two factors, x * f.y * f.x; NaN where a value is not finite.
__device__ __forceinline__ float2 inverse_norm(const Squares &s, float eps) {
    float scale = 1.f, sum = s.mid + s.small * (1.f / kSmallScale) * (1.f / kSmallScale);
    if (s.big > 0.f) {
        scale = kBigScale;
        sum = s.big + s.mid * kBigScale * kBigScale;
    } else if (s.mid == 0.f && s.small > 0.f) {
        scale = kSmallScale;
        sum = s.small;
    }
    if (!(sum < __int_as_float(0x7f800000))) return make_float2(__int_as_float(0x7fc00000), 1.f);
    return make_float2(1.f / (sqrtf(sum) + eps * scale), scale);
}

__device__ __forceinline__ Squares warp_squares(Squares s) {
    s.big = warp_sum(s.big);
    s.mid = warp_sum(s.mid);
    s.small = warp_sum(s.small);
    return s;
}

// The parts that a matrix's sum of squares is taken in.
int64_t parts_of(int64_t elements) { return std::min<int64_t>(592, (elements + 16383) / 16384); }

// A warp's unit of work: up to kSpan columns of a row.
constexpr int kSpan = 2048;

// Eight aligned elements as they lie in memory.
struct Eight {
    uint4 a, b;

    __device__ __forceinline__ void load(const char *row, int type, int64_t c) {
        if (type == OOP_TYPE_F32) {
            a = load_stream<OOP_TYPE_F32, 4>(reinterpret_cast<const float *>(row) + c).raw;
            b = load_stream<OOP_TYPE_F32, 4>(reinterpret_cast<const float *>(row) + c + 4).raw;
        } else {
            a = load_stream<OOP_TYPE_BF16, 8>(reinterpret_cast<const __nv_bfloat16 *>(row) + c).raw;
        }
    }
    __device__ __forceinline__ void get(int type, float (&v)[8]) const {
        if (type == OOP_TYPE_F32) {
            __builtin_memcpy(v, &a, 16);
            __builtin_memcpy(v + 4, &b, 16);
        } else {
            Packed<OOP_TYPE_BF16, 8> p;
            p.raw = a;
            p.get(v);
        }
    }
};

// use(values, column) for every eight columns of a warp's span, four loads ahead where the
// rows are aligned; columns from N on are 0.
template <class F>
__device__ __forceinline__ void each_eight(const char *row, int type, int64_t c0, int64_t end, int64_t N, bool wide, F &&use) {
    int64_t c = c0 + (threadIdx.x & 31) * 8;
    if (wide) {
        for (; c + 768 + 8 <= end; c += 1024) {
            Eight e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) e[k].load(row, type, c + 256 * k);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float v[8];
                e[k].get(type, v);
                use(v, c + 256 * k);
            }
        }
    }
    for (; c < end; c += 256) {
        float v[8];
        if (wide && c + 8 <= N) {
            Eight e;
            e.load(row, type, c);
            e.get(type, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = c + i < N ? load_any(row, type, c + i) : 0.f;
        }
        use(v, c);
    }
}

// Sum of squares of one part of each matrix (blockIdx.y).
__global__ void __launch_bounds__(256) squares_kernel(const char *x, int type, int64_t nb_row, int64_t nb_mat, int64_t N,
                                                      int64_t M, bool wide, Squares *sums) {
    __shared__ Squares part[8];
    let_next_start();
    const char *p = x + blockIdx.y * nb_mat;
    const int64_t spans = (N + kSpan - 1) / kSpan;
    Squares s;
    for (int64_t i = blockIdx.x * 8LL + (threadIdx.x >> 5); i < M * spans; i += gridDim.x * 8LL) {
        const int64_t r = i / spans, c0 = (i - r * spans) * kSpan, end = min(N, c0 + kSpan);
        each_eight(p + r * nb_row, type, c0, end, N, wide, [&](const float (&v)[8], int64_t) {
#pragma unroll
            for (int k = 0; k < 8; ++k) s.add(v[k]);
        });
    }
    s = warp_squares(s);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 8; ++i) {
            s.big += part[i].big;
            s.mid += part[i].mid;
            s.small += part[i].small;
        }
        sums[blockIdx.y * gridDim.x + blockIdx.x] = s;
    }
}

// X_0, scaled, as planes [2][B][M][pitch]; with DIRECT (no steps) scale * X_0 to y.
template <bool DIRECT>
__global__ void __launch_bounds__(256) start_kernel(const char *x, int type, int64_t nb_row, int64_t nb_mat, int64_t N, int64_t M,
                                                    bool wide, const Squares *sums, int parts, float eps, __half *dst, int64_t pitch,
                                                    char *y, int y_type, int64_t nb_y, int64_t nb_y_mat, float scale) {
    __shared__ float2 factors;
    let_next_start();
    wait_previous();
    if (threadIdx.x < 32) {
        Squares sum;
        for (int i = threadIdx.x; i < parts; i += 32) {
            const Squares one = sums[static_cast<int64_t>(blockIdx.y) * parts + i];
            sum.big += one.big;
            sum.mid += one.mid;
            sum.small += one.small;
        }
        sum = warp_squares(sum);
        if (threadIdx.x == 0) factors = inverse_norm(sum, eps);
    }
    __syncthreads();
    const float2 f = factors;
    const char *p = x + blockIdx.y * nb_mat;
    const int64_t plane = gridDim.y * M * pitch, spans = (N + kSpan - 1) / kSpan;
    for (int64_t i = blockIdx.x * 8LL + (threadIdx.x >> 5); i < M * spans; i += gridDim.x * 8LL) {
        const int64_t r = i / spans, c0 = (i - r * spans) * kSpan, end = min(N, c0 + kSpan);
        each_eight(p + r * nb_row, type, c0, end, N, wide, [&](float (&v)[8], int64_t c) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = v[k] * f.y * f.x;
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
        });
    }
}

// ---- few rows -------------------------------------------------------------
//
// A matrix whose smaller side n is at most 32 (an adapter's): all steps in one launch.  A
// cluster of up to eight CTAs holds X in shared memory as floats, each CTA a slice of the
// longer side; only the n x n partial products pass between them. Bound by latency: per
// step one exchange over the cluster, three barriers, and n^2 products per column, which
// the CUDA cores do faster than a tile of 256 rows could be loaded.  8 x 2560 in one
// launch instead of seventeen.

constexpr int kSmallCtas = 8;
constexpr int kSmallThreads = 256;

struct SmallArgs {
    const char *x;
    char *y;
    int64_t x_row, x_mat, y_row, y_mat;          // bytes
    int n, deep, slice, x_type, y_type, tall, steps;
    float eps, scale;
    float coefs[3 * kMaxSteps];
};

// Floats between columns of the slice: 16-byte units in odd number, so that neighbouring
// threads' columns lie in different banks.
__host__ __device__ constexpr int small_pitch(int nmax) { return nmax / 4 % 2 ? nmax : nmax + 4; }
constexpr size_t small_fixed_bytes(int nmax) {
    // every CTA's partial products (two steps'), the warps' parts, A and Q
    return static_cast<size_t>((2 * kSmallCtas + kSmallThreads / 32) * nmax * nmax + 2 * nmax * (nmax + 4)) * 4;
}
constexpr int small_columns(int nmax) {          // of a CTA, at most
    return static_cast<int>((kMostSmem - 2048 - small_fixed_bytes(nmax)) / (small_pitch(nmax) * 4));
}

__device__ __forceinline__ float load_float(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void store_float(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
template <int NMAX>
__global__ void __launch_bounds__(kSmallThreads) small_kernel(const __grid_constant__ SmallArgs a) {
    constexpr int kWarps = kSmallThreads / 32;
    constexpr int kPitch = small_pitch(NMAX), kSquare = NMAX * NMAX, kLd = NMAX + 4;
    constexpr int kGroups = 32 / NMAX;                     // columns of a warp at once
    extern __shared__ __align__(16) float small_smem[];
    __shared__ Squares reduce[32], my_sum;
    __shared__ float2 factors;
    float *partial = small_smem, *parts = partial + 2 * kSmallCtas * kSquare, *A = parts + kWarps * kSquare, *Q = A + NMAX * kLd;
    float *xs = Q + NMAX * kLd;
    const uint32_t cta = pair::cluster_rank(), ctas = pair::cluster_ctas();
    const int64_t matrix = blockIdx.x / ctas;
    const int s0 = static_cast<int>(cta) * a.slice, cols = max(0, min(a.slice, a.deep - s0));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const char *x = a.x + matrix * a.x_mat;
    char *y = a.y + matrix * a.y_mat;

    Squares sq;
    for (int i = tid; i < cols * (NMAX - a.n); i += kSmallThreads)               // rows that do not exist
        xs[i / (NMAX - a.n) * kPitch + a.n + i % (NMAX - a.n)] = 0.f;
    auto take = [&](int r, int s, float v) {
        sq.add(v);
        xs[s * kPitch + r] = v;
    };
    constexpr int kAhead = 8;                              // loads before the first is used
    if (a.tall) {                                          // lanes along the rows, which are short
        const int total = cols * a.n;
        for (int i0 = tid; i0 < total; i0 += kSmallThreads * kAhead) {
            float v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + k * kSmallThreads, s = i / a.n;
                v[k] = i < total ? load_any(x + static_cast<int64_t>(s0 + s) * a.x_row, a.x_type, i - s * a.n) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + k * kSmallThreads, s = i / a.n;
                if (i < total) take(i - s * a.n, s, v[k]);
            }
        }
    } else {                                               // a row to a warp
        for (int r = warp; r < a.n; r += kWarps)
            for (int c0 = lane; c0 < cols; c0 += 32 * kAhead) {
                float v[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    v[k] = c0 + 32 * k < cols ? load_any(x + r * a.x_row, a.x_type, s0 + c0 + 32 * k) : 0.f;
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (c0 + 32 * k < cols) take(r, c0 + 32 * k, v[k]);
            }
    }
    sq = warp_squares(sq);
    if (lane == 0) reduce[warp] = sq;
    __syncthreads();
    if (warp == 0) {
        sq = warp_squares(lane < kWarps ? reduce[lane] : Squares());
        if (lane == 0) my_sum = sq;
    }
    if (ctas > 1) {
        pair::cluster_sync();
        if (warp == 0) {                                   // a lane reads a CTA's
            Squares s;
            if (lane < ctas) {
                const uint32_t at = pair::cluster_addr(&my_sum, lane);
                s.big = load_float(at);
                s.mid = load_float(at + 4);
                s.small = load_float(at + 8);
            }
            sq = warp_squares(s);
        }
    }
    if (tid == 0) factors = inverse_norm(sq, a.eps);
    __syncthreads();
    const float2 f = factors;
    for (int i = tid; i < cols * NMAX; i += kSmallThreads) {
        float &v = xs[i / NMAX * kPitch + i % NMAX];
        v = v * f.y * f.x;
    }
    for (int step = 0; step < a.steps; ++step) {
        __syncthreads();
        // products of rows over this CTA's columns: a lane's row with every row
        float acc[NMAX];
#pragma unroll
        for (int j = 0; j < NMAX; ++j) acc[j] = 0.f;
        const int row = lane % NMAX, group = lane / NMAX;
#pragma unroll 4
        for (int s = warp * kGroups + group; s < cols; s += kWarps * kGroups) {
            const float *c = xs + s * kPitch;
            const float own = c[row];
#pragma unroll
            for (int j = 0; j < NMAX; j += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(c + j);
                acc[j] = fmaf(own, v.x, acc[j]);
                acc[j + 1] = fmaf(own, v.y, acc[j + 1]);
                acc[j + 2] = fmaf(own, v.z, acc[j + 2]);
                acc[j + 3] = fmaf(own, v.w, acc[j + 3]);
            }
        }
#pragma unroll
        for (int o = NMAX; o < 32; o <<= 1)
#pragma unroll
            for (int j = 0; j < NMAX; ++j) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
        if (group == 0) {
#pragma unroll
            for (int j = 0; j < NMAX; ++j) parts[warp * kSquare + j * NMAX + row] = acc[j];
        }
        __syncthreads();
        // sent to every CTA as they are ready; two steps' apart, as a slow CTA may still read the
        // last one's
        float *all = partial + (step & 1) * kSmallCtas * kSquare;
        for (int e = tid; e < kSquare; e += kSmallThreads) {
            float v = 0.f;
#pragma unroll
            for (int p = 0; p < kWarps; ++p) v += parts[p * kSquare + e];
            for (uint32_t c = 0; c < ctas; ++c) store_float(pair::cluster_addr(all + cta * kSquare + e, c), v);
        }
        if (ctas > 1) pair::cluster_sync();
        else __syncthreads();
        for (int e = tid; e < kSquare; e += kSmallThreads) {
            float v = 0.f;
#pragma unroll
            for (uint32_t c = 0; c < kSmallCtas; ++c)
                if (c < ctas) v += all[c * kSquare + e];
            A[e / NMAX * kLd + e % NMAX] = v;
        }
        __syncthreads();
        const float *co = a.coefs + 3 * step;
        for (int e = tid; e < kSquare; e += kSmallThreads) {
            const int i = e / NMAX, j = e % NMAX;
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < NMAX; k += 4) {
                const float4 p = *reinterpret_cast<const float4 *>(A + i * kLd + k), q = *reinterpret_cast<const float4 *>(A + j * kLd + k);
                v = fmaf(p.x, q.x, fmaf(p.y, q.y, fmaf(p.z, q.z, fmaf(p.w, q.w, v))));
            }
            Q[i * kLd + j] = fmaf(co[2], v, fmaf(co[1], A[i * kLd + j], i == j ? co[0] : 0.f));
        }
        __syncthreads();
        for (int s = tid; s < cols; s += kSmallThreads) {
            float *c = xs + s * kPitch, v[NMAX];
#pragma unroll
            for (int j = 0; j < NMAX; j += 4) {
                const float4 w = *reinterpret_cast<const float4 *>(c + j);
                v[j] = w.x, v[j + 1] = w.y, v[j + 2] = w.z, v[j + 3] = w.w;
            }
#pragma unroll(NMAX > 8 ? 1 : 2)
            for (int i0 = 0; i0 < NMAX; i0 += 4) {
                float4 out;
                float *o = &out.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
                    for (int j = 0; j < NMAX; j += 4) {
                        const float4 q = *reinterpret_cast<const float4 *>(Q + (i0 + i) * kLd + j);
                        sum0 = fmaf(q.x, v[j], fmaf(q.y, v[j + 1], sum0));
                        sum1 = fmaf(q.z, v[j + 2], fmaf(q.w, v[j + 3], sum1));
                    }
                    o[i] = sum0 + sum1;
                }
                *reinterpret_cast<float4 *>(c + i0) = out;
            }
        }
    }
    __syncthreads();
    auto put = [&](char *row, int64_t at, float v) {
        if (a.y_type == OOP_TYPE_F32) reinterpret_cast<float *>(row)[at] = a.scale * v;
        else reinterpret_cast<__nv_bfloat16 *>(row)[at] = __float2bfloat16_rn(a.scale * v);
    };
    if (a.tall) {
        for (int i = tid; i < cols * a.n; i += kSmallThreads) {
            const int s = i / a.n, r = i - s * a.n;
            put(y + static_cast<int64_t>(s0 + s) * a.y_row, r, xs[s * kPitch + r]);
        }
    } else {
        for (int r = warp; r < a.n; r += kWarps)
#pragma unroll 4
            for (int c = lane; c < cols; c += 32) put(y + r * a.y_row, s0 + c, xs[c * kPitch + r]);
    }
    if (ctas > 1) pair::cluster_sync();                          // no CTA ends while another reads its sums
}

// CTAs of a matrix's cluster, 0 where it has to go the other way: by its size alone.
int small_ctas(int64_t n, int64_t deep) {
    if (n > 32) return 0;
    const int nmax = n <= 8 ? 8 : n <= 16 ? 16 : 32;
    // 128 columns to a CTA: fewer would not shorten the step, whose exchange takes 1300 cycles
    int ctas = 1;
    while (ctas < kSmallCtas && deep > 128LL * ctas) ctas *= 2;
    return deep <= static_cast<int64_t>(small_columns(nmax)) * ctas ? ctas : 0;
}

template <int NMAX>
cudaError_t launch_small(const SmallArgs &a, int ctas, int64_t matrices, cudaStream_t st) {
    cudaError_t e = allow_smem<small_kernel<NMAX>>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas * matrices));
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = small_fixed_bytes(NMAX) + static_cast<size_t>(a.slice) * small_pitch(NMAX) * 4;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    ++g_kernel_launches;
    return cudaLaunchKernelEx(&cfg, small_kernel<NMAX>, a);
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

size_t plane_pair_bytes(int64_t cols, int64_t rows, int64_t B) {
    return pair::round256(static_cast<size_t>(2 * B * rows * pair::round8(cols)) * 2);
}

// The tiles of A = X X': those that would leave SMs idle go in parts of k (200 x 2560 is
// one tile of 40 stages, 32 us).
pair::TileMap map_of_a(int64_t n, int64_t deep, int64_t B) {
    return pair::tile_map(n, n, 256, (deep + pair::kDepth - 1) / pair::kDepth, 3, B, true, true);
}

// About the time of a product in microseconds: 9 for a launch, 0.8 for each stage of a
// wave of tiles, 6 for the join of parts.
double product_time(int64_t tiles, int64_t k, int parts) {
    const int64_t blocks = (k + pair::kDepth - 1) / pair::kDepth, waves = tiles / pair::kPairs;
    const int64_t last = tiles % pair::kPairs ? (blocks + parts - 1) / parts : 0;
    return 9.0 + 0.8 * static_cast<double>(waves * blocks + last) + (parts > 1 ? 6.0 : 0.0);
}

// B matrices of two planes: [2][B][rows][pitch].
struct Planes {
    char *p;
    int64_t cols, rows, B;
    int64_t pitch() const { return pair::round8(cols); }
    int64_t matrix_bytes() const { return rows * pitch() * 2; }
    __half *hi() const { return reinterpret_cast<__half *>(p); }
    __half *lo() const { return reinterpret_cast<__half *>(p + B * matrix_bytes()); }
    pair::Operand operand(bool rows_contiguous) const {
        return {p, cols, rows, pitch() * 2, matrix_bytes(), 2 * B, rows_contiguous, true};
    }
};

// Steps on A alone.  Q is a polynomial of A, so X_s = Z X_0 with Z <- Q Z, A <- Q A Q: all
// products but the first and the last are of the smaller side alone, 3 r + 5 s - 4 of them
// (in n^3, symmetric results counted half) against s (3 r + 1) for a matrix r times as
// long as wide: fewer from r = 4/3 on, but more launches.  Z is symmetric as a polynomial,
// but not as computed, and is kept whole: Q's rounding meets the small singular values'
// large factors on one side of Q Z alone, and half of it mirrored would bring them to the
// leading ones (an update of rank one was off by 11%).  What is left is the loss of
// precision in A: a rounding of it grows by Q^2 at every step, where one of X grows by Q,
// and reaches the last Q as this share of it.  So only results of 16 bits are computed this
// way, and only where the share stays below their rounding (five steps of the usual
// coefficients: measured up to 4096 x 12288, 1.3e-3 of the result's norm for an update of
// rank one, below 4e-4 for others; bfloat16's own rounding is 1.7e-3).
//
// The eigenvalues l of A start within 0 .. 1, and a step takes them to l q(l)^2, with q(l) =
// a + b l + c l^2: the largest magnitudes of q and of its slope, and the slope of l q^2
// (what a rounding grows by), are taken over the range that the steps so far can reach.
struct Reach {
    double top = 1.0, z = 1.0;     // of the eigenvalues, of Z's
    double grown = 0x1p-24;        // a rounding of A
    double share = 0.0;            // of the Qs so far
    void step(const float *c) {
        double q_most = 0.0, slope_most = 0.0, growth = 0.0, next = 0.0;
        for (int i = 0; i <= 64; ++i) {
            const double l = top * i / 64.0, q = c[0] + l * (c[1] + l * c[2]), slope = c[1] + 2.0 * l * c[2];
            q_most = std::max(q_most, std::fabs(q));
            slope_most = std::max(slope_most, std::fabs(slope));
            growth = std::max({growth, q * q, std::fabs(q * q + 2.0 * l * q * slope)});
            next = std::max(next, l * q * q);
        }
        share += grown * slope_most / std::max(1e-3, std::fabs(static_cast<double>(c[0])));
        grown = std::max(grown * growth, 0x1p-24);
        z *= q_most;
        top = 1.01 * next;                                 // between the samples
    }
};
bool on_a_alone(int64_t n, int64_t deep, int64_t B, int steps, const float *coefs) {
    if (steps < 2) return false;
    Reach r;
    for (int i = 0; i < steps; ++i) r.step(coefs ? coefs + 3 * i : kDefault);
    if (!(r.share <= 0x1p-9 && r.z <= 0x1p20)) return false;               // and Z keeps 19 bits of its leading part
    const int64_t t = (n + 255) / 256, half = t * (t + 1) / 2 * B, whole = t * ((deep + 255) / 256) * B;
    const double first = product_time(half, deep, map_of_a(n, deep, B).parts), square = product_time(half, n, 1), with_x = product_time(whole, n, 1);
    const double whole_z = product_time(t * t * B, n, 1);
    return first + (3 * steps - 2) * square + (steps - 1) * whole_z + with_x < steps * (first + square + with_x);
}

// The tiles of A in parts: summed, scaled, with the shift on the diagonal, as planes.
__global__ void __launch_bounds__(256) join_kernel(const pair::TileMap map, const float *slots, int64_t n, int64_t pitch, float alpha,
                                                   float diag, __half *hi, __half *lo) {
    let_next_start();
    wait_previous();
    pair::each_joined<256>(map, slots, [&](int z, int64_t r, int64_t c, float4 v) {
        if (r >= n) return;
        const float f[4] = {v.x, v.y, v.z, v.w};
        const int64_t at = (z * n + r) * pitch + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (c + i >= n) continue;
            const float one = f[i] * alpha + (r == c + i ? diag : 0.f);
            hi[at + i] = __float2half_rn(one);
            lo[at + i] = __float2half_rn(one - __half2float(hi[at + i]));
        }
    });
}

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
    s.result = d.operand(false);
    s.out.nb0 = d.pitch() * 2;
    s.out.batch = d.matrix_bytes();
    s.out.planes = static_cast<int>(d.B);
    s.out.alpha = alpha;
}

}  // namespace
}  // namespace oop

using namespace oop;

extern "C" {

size_t oop_orthogonalise_workspace_size(const int64_t ne[3]) {
    if (check_sizes(ne) != OOP_OK || ne[0] == 0 || ne[1] == 0 || ne[2] == 0) return 0;
    const int64_t n = std::min(ne[0], ne[1]);
    if (small_ctas(n, std::max(ne[0], ne[1]))) return 0;
    const size_t x = plane_pair_bytes(ne[0], ne[1], ne[2]), a = plane_pair_bytes(n, n, ne[2]);
    return pair::round256(static_cast<size_t>(ne[2] * parts_of(ne[0] * ne[1])) * sizeof(Squares)) + std::max(2 * x + 2 * a, x + 5 * a) +
           pair::slot_bytes(map_of_a(n, std::max(ne[0], ne[1]), ne[2]), ne[2], 256);
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
    const int64_t n = std::min(M, N), deep = std::max(M, N);
    const bool tall = M > N;
    const int ctas = small_ctas(n, deep);
    if (!ctas && (!workspace || workspace_bytes < oop_orthogonalise_workspace_size(ne) || !is_aligned(workspace, 256)))
        return OOP_ERR_WORKSPACE;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (ctas) {
        SmallArgs a = {};
        a.x = static_cast<const char *>(x);
        a.y = static_cast<char *>(y);
        a.x_row = nb_x[0], a.x_mat = nb_x[1], a.y_row = nb_y[0], a.y_mat = nb_y[1];
        a.n = static_cast<int>(n);
        a.deep = static_cast<int>(deep);
        a.slice = static_cast<int>((deep + ctas - 1) / ctas);
        a.x_type = x_type, a.y_type = y_type, a.tall = tall, a.steps = steps;
        a.eps = eps, a.scale = scale;
        for (int i = 0; i < 3 * steps; ++i) a.coefs[i] = coefs ? coefs[i] : kDefault[i % 3];
        const cudaError_t e = n <= 8    ? launch_small<8>(a, ctas, B, st)
                              : n <= 16 ? launch_small<16>(a, ctas, B, st)
                                        : launch_small<32>(a, ctas, B, st);
        return cuda_status(e);
    }
    const int parts = static_cast<int>(parts_of(M * N));
    Squares *sums = static_cast<Squares *>(workspace);
    char *at = static_cast<char *>(workspace) + pair::round256(static_cast<size_t>(B * parts) * sizeof(Squares));
    Planes X = {at, N, M, B}, next = {at + plane_pair_bytes(N, M, B), N, M, B};
    const Planes A = {next.p + plane_pair_bytes(N, M, B), n, n, B}, Q = {A.p + plane_pair_bytes(n, n, B), n, n, B};
    const char *xp = static_cast<const char *>(x);
    char *yp = static_cast<char *>(y);
    const unsigned nb = static_cast<unsigned>(B);
    const bool wide = is_aligned(x, 16) && (M <= 1 || nb_x[0] % 16 == 0) && (B <= 1 || nb_x[1] % 16 == 0);
    const int64_t units = M * ((N + kSpan - 1) / kSpan);
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((units + 7) / 8, 1216));
    squares_kernel<<<dim3(static_cast<unsigned>(parts), nb), 256, 0, st>>>(xp, x_type, nb_x[0], nb_x[1], N, M, wide, sums);
    auto start = [&](auto kernel, __half *planes, int64_t pitch) {
        return launch_dependent(kernel, dim3(blocks, nb), 256, 0, st, xp, x_type, nb_x[0], nb_x[1], N, M, wide,
                                static_cast<const Squares *>(sums), parts, eps, planes, pitch, yp, y_type, nb_y[0], nb_y[1], scale);
    };
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = steps == 0 ? start(start_kernel<true>, nullptr, 0) : start(start_kernel<false>, X.hi(), X.pitch());
    g_kernel_launches = 2;
    // A = X X', or X' X, with a shift in its diagonal
    float *slots = reinterpret_cast<float *>(
        X.p + std::max(2 * plane_pair_bytes(N, M, B) + 2 * plane_pair_bytes(n, n, B), plane_pair_bytes(N, M, B) + 5 * plane_pair_bytes(n, n, B)));
    const pair::TileMap map = map_of_a(n, deep, B);
    auto square_of = [&](const Planes &x_now, const Planes &d, double shift) {
        constexpr float kAlpha = kScaleA / (kScaleX * kScaleX);
        const float diag = static_cast<float>(shift * kScaleA);
        pair::Spec p = product_of(x_now, tall, x_now, tall, n, n, deep);
        p.symmetric = true;
        p.in_parts = true;
        p.out.slots = slots;
        to_planes(p, d, kAlpha);
        p.out.diag = diag;
        const cudaError_t err = pair::launch<pair::kSplit, true, 256>(p, status, st);
        if (err != cudaSuccess || map.parts == 1) return err;
        ++g_kernel_launches;
        return launch_dependent(join_kernel, dim3(static_cast<unsigned>(pair::kJoinCtas * pair::tiles_in_parts(map, B))), 256, 0, st, map,
                                static_cast<const float *>(slots), n, d.pitch(), kAlpha, diag, d.hi(), d.lo());
    };
    auto last_product = [&](pair::Spec p, float alpha) {
        p.out.p0 = yp;
        p.out.nb0 = nb_y[0];
        p.out.batch = nb_y[1];
        p.out.type = y_type;
        p.out.alpha = alpha;                               // a power of two: its product with a small scale would lose bits
        p.out.beta = scale;
        p.out.wide = N * ys % 16 == 0 && is_aligned(y, 16) && (M <= 1 || nb_y[0] % 16 == 0) && (B <= 1 || nb_y[1] % 16 == 0);
        return pair::launch<pair::kPlain, true, 256>(p, status, st);
    };
    if (e == cudaSuccess && y_type == OOP_TYPE_BF16 && on_a_alone(n, deep, B, steps, coefs)) {
        Planes pool[4], Z = {}, P = Q;                     // beside A: P, Q, Z and the next Z
        for (int i = 0; i < 4; ++i) pool[i] = {next.p + (1 + i) * plane_pair_bytes(n, n, B), n, n, B};
        const Planes G = {next.p, n, n, B};                // A
        int free_ones[3] = {1, 2, 3};                      // pool[0] is P's
        P = pool[0];
        double z_scale = 1.0;
        Reach reach;                                       // Z's planes leave room for what it can reach
        pair::Spec s;
        e = square_of(X, G, 0.0);
        auto symmetric = [&](const Planes &a, const Planes &b, const Planes &d, double alpha) {
            s = product_of(a, false, b, false, n, n, n);
            s.symmetric = s.a_half = s.b_half = true;
            to_planes(s, d, static_cast<float>(alpha));
        };
        int z_at = -1;
        for (int i = 0; i < steps && e == cudaSuccess; ++i) {
            const float *c = coefs ? coefs + 3 * i : kDefault;
            int q_at = -1;
            for (int k : free_ones)
                if (k != z_at && q_at < 0) q_at = k;
            const Planes q = pool[q_at];
            symmetric(G, G, q, c[2] * (kScaleQ / (kScaleA * kScaleA)));        // Q = a + b A + c A A
            s.out.c_hi = G.hi();
            s.out.c_lo = G.lo();
            s.out.beta = c[1] * (kScaleQ / kScaleA);
            s.out.diag = c[0] * kScaleQ;
            e = pair::launch<pair::kSplit, true, 256>(s, status, st);
            reach.step(c);
            if (i == 0) {
                z_at = q_at;
                z_scale = kScaleQ;
            } else if (e == cudaSuccess) {                 // Z <- Q Z
                int to = -1;
                for (int k : free_ones)
                    if (k != z_at && k != q_at) to = k;
                const double next_scale = std::exp2(std::floor(std::log2(32768.0 / std::max(reach.z, 1.0))));
                s = product_of(q, false, pool[z_at], i > 1, n, n, n);              // whole from here on; the first was a Q
                s.a_half = true;
                s.b_half = i == 1;
                to_planes(s, pool[to], static_cast<float>(next_scale / (kScaleQ * z_scale)));
                e = pair::launch<pair::kSplit, true, 256>(s, status, st);
                z_scale = next_scale;
                z_at = to;
            }
            if (i + 1 < steps && e == cudaSuccess) {       // A <- Q A Q
                symmetric(G, q, P, 1.0 / kScaleQ);
                e = pair::launch<pair::kSplit, true, 256>(s, status, st);
                symmetric(P, q, G, 1.0 / kScaleQ);
                if (e == cudaSuccess) e = pair::launch<pair::kSplit, true, 256>(s, status, st);
            }
        }
        if (e != cudaSuccess) return cuda_status(e);
        Z = pool[z_at];
        s = tall ? product_of(X, false, Z, false, M, N, N) : product_of(Z, false, X, true, M, N, M);   // X_0 Z', or Z X_0
        return cuda_status(last_product(s, static_cast<float>(1.0 / (z_scale * kScaleX))));
    }
    for (int i = 0; i < steps && e == cudaSuccess; ++i) {
        const float *c = coefs ? coefs + 3 * i : kDefault;
        // a + b A + c A A = c (A + b / 2c)^2 + a - b^2 / 4c: with the shift in A's diagonal Q is
        // one product, and A need not be read again.  The shift has to be of A's size, and to bring
        // A's eigenvalues, which are not negative, closer to 0: A's planes have no room above 64.
        const bool square = c[2] != 0.f && (c[1] == 0.f || (c[1] < 0.f) != (c[2] < 0.f)) && std::fabs(c[1]) <= 8.f * std::fabs(c[2]);
        const double shift = square ? 0.5 * c[1] / c[2] : 0.0;
        e = square_of(X, A, shift);
        if (e != cudaSuccess) break;
        pair::Spec s = product_of(A, false, A, false, n, n, n);                           // Q = a + b A + c A A
        s.symmetric = s.a_half = s.b_half = true;
        to_planes(s, Q, c[2] * (kScaleQ / (kScaleA * kScaleA)));
        s.out.diag = static_cast<float>((c[0] - c[2] * shift * shift) * kScaleQ);
        if (!square) {
            s.out.c_hi = A.hi();
            s.out.c_lo = A.lo();
            s.out.beta = c[1] * (kScaleQ / kScaleA);
        }
        e = pair::launch<pair::kSplit, true, 256>(s, status, st);
        if (e != cudaSuccess) break;
        s = tall ? product_of(X, false, Q, false, M, N, N) : product_of(Q, false, X, true, M, N, M);   // X Q, or Q X
        s.a_half = !tall;
        s.b_half = tall;
        if (i + 1 < steps) {
            to_planes(s, next, 1.f / kScaleQ);
            e = pair::launch<pair::kSplit, true, 256>(s, status, st);
        } else {
            e = last_product(s, 1.f / (kScaleQ * kScaleX));
        }
        std::swap(X, next);
    }
    return cuda_status(e);
}

}  // extern "C"
