// gated_ffn.cu -- the gated feed-forward block up to its last projection, and its backward
// pass.
//
//   gate = x Wg',  up = x Wu',  h = act(gate) up
//   dgate = dh up act'(gate),  dup = dh act(gate)
//   dx = dgate Wg + dup Wu,  dWg = dgate' x,  dWu = dup' x
//
// Bound by the tensor cores from a few hundred tokens on.  Forward: one product whose
// tiles take half their columns from each weight, so that a tile's epilogue holds the
// gates and the ups of the same features and nothing goes to memory between.  Backward:
// one pass over dh, gate and up writes dgate and dup (16 bits each where dh has 16), then
// dx as one product over both weights' rows, and both weight gradients as one product of
// two batches; the operands lie as they are, with their rows or their k contiguous.
//
// Measured: bf16 8192 x 5120 x 17408, gate and up kept: 1.53 ms, 1.91 PFLOP/s (97% of the
// measured burst of cuBLAS), 1.79 to 1.89 ms a call where the card's power limit holds;
// backward 8192 x 2560 x 9728: 1.02 to 1.07 ms, 1.52 to 1.60 PFLOP/s, 0.13 or more of it for
// dgate and dup.  f32 512 x 2560 x 9728, kept: 165 us, 60 of it for the planes of the weights, the
// rest two waves of tiles with their epilogues.
#include <algorithm>
#include <cmath>

#include "activation.cuh"
#include "oop_internal.cuh"
#include "pair_product.cuh"
#include "quant.cuh"
#include "rows.cuh"

namespace oop {
namespace {

// The nearest bfloat16; a finite value stays finite.
__device__ __forceinline__ __nv_bfloat16 nearest_bf16(float v) {
    const float top = __uint_as_float(0x7f7f0000u);        // the largest one
    return __float2bfloat16_rn(isfinite(v) ? fminf(fmaxf(v, -top), top) : v);
}

// v as the sum of P bfloat16 values, each the nearest to what is left.
template <int P>
__device__ __forceinline__ void split(float v, __nv_bfloat16 (&t)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        t[i] = nearest_bf16(v);
        v -= __bfloat162float(t[i]);
    }
}

// Eight aligned elements of a plain type as they lie in memory: the load alone, so that
// several can be in flight.
template <int TYPE>
struct Eight {
    static constexpr int E = 16 / plain_size(TYPE);
    Packed<TYPE, E> part[8 / E];

    __device__ __forceinline__ void load(const char *row, int64_t c) {
        const auto *p = reinterpret_cast<const typename Plain<TYPE>::S *>(row) + c;
#pragma unroll
        for (int i = 0; i < 8 / E; ++i) part[i] = load_stream<TYPE, E>(p + i * E);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8 / E; ++i) {
            float f[E];
            part[i].get(f);
#pragma unroll
            for (int k = 0; k < E; ++k) v[i * E + k] = f[k];
        }
    }
};

// Eight elements of a row from column c, those beyond the row 0.
template <int TYPE>
__device__ __forceinline__ void load8(const char *row, int64_t c, int64_t cols, int wide, float (&v)[8]) {
    if constexpr (plain_size(TYPE) != 0) {
        using S = typename Plain<TYPE>::S;
        const S *p = reinterpret_cast<const S *>(row) + c;
        if (wide && c + 8 <= cols) {
            Eight<TYPE> e;
            e.load(row, c);
            e.get(v);
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? to_float(p[i]) : 0.f;
    } else {                                               // whole blocks: cols % 32 == 0
        using F = QFormat<TYPE>;
        const uint8_t *blk = reinterpret_cast<const uint8_t *>(row) + c / F::QK * F::BYTES;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = decode<TYPE>(blk, static_cast<int>(c % F::QK) + i);
    }
}

template <int P>
__device__ __forceinline__ void store_planes(const float (&v)[8], __nv_bfloat16 *dst, int64_t plane) {
    __nv_bfloat16 t[P][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        __nv_bfloat16 one[P];
        split<P>(v[i], one);
#pragma unroll
        for (int p = 0; p < P; ++p) t[p][i] = one[p];
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
        uint4 w;
        __builtin_memcpy(&w, t[p], 16);
        *reinterpret_cast<uint4 *>(dst + p * plane) = w;
    }
}

// Rows of any type as P bfloat16 planes [P][rows][pitch]; P = 0: 16-bit elements copied.
template <int TYPE, int P>
__global__ void __launch_bounds__(256) planes_kernel(const char *src, int64_t nb, int64_t cols, int64_t rows,
                                                     __nv_bfloat16 *dst, int64_t pitch, int wide) {
    const int64_t per_row = pitch / 8;
    let_next_start();
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < rows * per_row; i += gridDim.x * 256LL) {
        const int64_t r = i / per_row, c = (i - r * per_row) * 8;
        if constexpr (P == 0) {
            uint16_t w[8];
            const uint16_t *p = reinterpret_cast<const uint16_t *>(src + r * nb) + c;
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = c + k < cols ? p[k] : 0;
            uint4 o;
            __builtin_memcpy(&o, w, 16);
            *reinterpret_cast<uint4 *>(dst + r * pitch + c) = o;
        } else {
            float v[8];
            load8<TYPE>(src + r * nb, c, cols, wide, v);
            store_planes<P>(v, dst + r * pitch + c, rows * pitch);
        }
    }
}

unsigned blocks_of(int64_t n) { return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((n + 255) / 256, 1 << 16))); }

template <int P>
cudaError_t launch_planes_of(const void *src, int type, int64_t nb, int64_t cols, int64_t rows, void *dst, int64_t pitch,
                             cudaStream_t st) {
    const char *s = static_cast<const char *>(src);
    auto *d = static_cast<__nv_bfloat16 *>(dst);
    const int wide = is_aligned(src, 16) && nb % 16 == 0;
    const unsigned g = blocks_of(rows * pitch / 8);
#define OOP_CASE(T) \
    case T: planes_kernel<T, P><<<g, 256, 0, st>>>(s, nb, cols, rows, d, pitch, wide); break;
    if constexpr (P == 0) {
        planes_kernel<OOP_TYPE_BF16, 0><<<g, 256, 0, st>>>(s, nb, cols, rows, d, pitch, wide);
    } else {
        switch (type) {
            OOP_CASE(OOP_TYPE_F32) OOP_CASE(OOP_TYPE_F16) OOP_CASE(OOP_TYPE_Q4_0)
            OOP_CASE(OOP_TYPE_Q4_1) OOP_CASE(OOP_TYPE_Q5_0) OOP_CASE(OOP_TYPE_Q5_1) OOP_CASE(OOP_TYPE_Q8_0)
            OOP_CASE(OOP_TYPE_Q2_K) OOP_CASE(OOP_TYPE_Q3_K) OOP_CASE(OOP_TYPE_Q4_K) OOP_CASE(OOP_TYPE_Q5_K)
            OOP_CASE(OOP_TYPE_Q6_K)
        }
    }
#undef OOP_CASE
    ++g_kernel_launches;
    return cudaGetLastError();
}

// ---- few tokens -----------------------------------------------------------
//
// Up to eight tokens: the weights' bytes are all there is to do, and the tensor cores'
// tiles of 256 tokens would only be waited for.  A warp takes a feature: its gate and its
// up row, each read once in long runs (five or six 16-byte loads of each row in flight per
// lane), against the tokens in shared memory as floats.  Sums in fp32 on the CUDA cores,
// which any type of weight allows without a copy.  bf16, 1 x 2560 x 9728: 17.7 us, 5.6
// TB/s, 84% of the measured copy rate (one load of each row at a time: 48 us; on the
// tensor cores 44 us).
constexpr int kFewThreads = 512, kFewTokens = 8;
constexpr int64_t kFewBytes = 180 * 1024;

struct FewArgs {
    const char *x, *w[2];
    char *h, *gate, *up;
    int64_t nb_x, nb_w, nb_h, nb_gu, K, F;
    int T, x_type, act, wide;
};

template <int TYPE, int NT>
__global__ void __launch_bounds__(kFewThreads, 1) few_kernel(const __grid_constant__ FewArgs a) {
    // x by eights: the first four of each eight of all tokens, then the last four, so that
    // neighbouring lanes read neighbouring 16 bytes
    extern __shared__ __align__(16) float few_x[];
    const int64_t eights = (a.K + 7) / 8, half = eights * 4;
    for (int64_t i = threadIdx.x; i < NT * eights * 8; i += kFewThreads) {
        const int64_t t = i / (eights * 8), k = i - t * eights * 8;
        const float v = t < a.T && k < a.K ? load_any(a.x + t * a.nb_x, a.x_type, k) : 0.f;
        few_x[(t * 2 + (k >> 2 & 1)) * half + (k >> 3) * 4 + (k & 3)] = v;
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t f = blockIdx.x * (kFewThreads / 32) + warp; f < a.F; f += gridDim.x * (kFewThreads / 32)) {
        uint64_t acc[2][NT] = {};                          // pairs: even and odd columns
        const char *row[2] = {a.w[0] + f * a.nb_w, a.w[1] + f * a.nb_w};
        auto add = [&](const float (&w)[2][8], int64_t e) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float4 v = *reinterpret_cast<const float4 *>(few_x + (t * 2 + q) * half + e * 4);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        acc[r][t] = ptx::fma2(ptx::pack2(w[r][4 * q], w[r][4 * q + 1]), ptx::pack2(v.x, v.y), acc[r][t]);
                        acc[r][t] = ptx::fma2(ptx::pack2(w[r][4 * q + 2], w[r][4 * q + 3]), ptx::pack2(v.z, v.w), acc[r][t]);
                    }
                }
            }
        };
        int64_t e = lane;
        if constexpr (plain_size(TYPE) != 0) {
            constexpr int kAhead = TYPE == OOP_TYPE_F32 ? 3 : 5;
            for (; a.wide && e - lane + 32 * kAhead <= a.K / 8; e += 32 * kAhead) {
                Eight<TYPE> raw[kAhead][2];
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
#pragma unroll
                    for (int r = 0; r < 2; ++r) raw[k][r].load(row[r], (e + 32 * k) * 8);
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    float w[2][8];
                    raw[k][0].get(w[0]);
                    raw[k][1].get(w[1]);
                    add(w, e + 32 * k);
                }
            }
        }
        for (; e < eights; e += 32) {
            float w[2][8];
            load8<TYPE>(row[0], e * 8, a.K, a.wide, w[0]);
            load8<TYPE>(row[1], e * 8, a.K, a.wide, w[1]);
            add(w, e);
        }
        float g = 0.f, u = 0.f;                            // lane t: token t's
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float lo, hi;
            ptx::unpack2(acc[0][t], lo, hi);
            const float gt = warp_sum(lo + hi);
            ptx::unpack2(acc[1][t], lo, hi);
            const float ut = warp_sum(lo + hi);
            if (lane == t) g = gt, u = ut;
        }
        if (lane >= a.T) continue;
        auto put = [&](char *p, int64_t nb, float v) {
            char *row = p + lane * nb;
            if (a.x_type == OOP_TYPE_F32) reinterpret_cast<float *>(row)[f] = v;
            else if (a.x_type == OOP_TYPE_F16) reinterpret_cast<__half *>(row)[f] = __float2half_rn(v);
            else reinterpret_cast<__nv_bfloat16 *>(row)[f] = __float2bfloat16_rn(v);
        };
        put(a.h, a.nb_h, activation_of(a.act, g) * u);
        if (a.gate) {
            put(a.gate, a.nb_gu, g);
            put(a.up, a.nb_gu, u);
        }
    }
}

// Operands that the tensor cores take as they are go there from five tokens on (bf16 5120 x
// 17408: 4 tokens 77 us here and 91 there, 5 tokens 126 and 83), others have to be copied
// first (f32: 8 tokens 162 us here and 488 there).
bool few_tokens(int64_t T, int64_t K, int x_type, int w_type) {
    const int64_t nt = !plain_size(w_type) ? 8 : T <= 1 ? 1 : T <= 2 ? 2 : T <= 4 ? 4 : 8;
    const bool native = x_type == w_type && plain_size(w_type) == 2;
    return T <= (native ? 4 : kFewTokens) && nt * ((K + 7) / 8) * 32 <= kFewBytes;
}

template <int TYPE, int NT>
cudaError_t launch_few(const FewArgs &a, cudaStream_t st) {
    const cudaError_t e = allow_smem<few_kernel<TYPE, NT>>();
    if (e != cudaSuccess) return e;
    const int64_t per = kFewThreads / 32, ctas = std::min<int64_t>((a.F + per - 1) / per, device_sm_count());
    few_kernel<TYPE, NT><<<static_cast<unsigned>(ctas), kFewThreads, static_cast<size_t>(NT * ((a.K + 7) / 8) * 32), st>>>(a);
    ++g_kernel_launches;
    return cudaGetLastError();
}
template <int TYPE>
cudaError_t launch_few(const FewArgs &a, cudaStream_t st) {
    if constexpr (plain_size(TYPE) != 0) {
        if (a.T <= 1) return launch_few<TYPE, 1>(a, st);
        if (a.T <= 2) return launch_few<TYPE, 2>(a, st);
        if (a.T <= 4) return launch_few<TYPE, 4>(a, st);
    }
    return launch_few<TYPE, 8>(a, st);
}
cudaError_t launch_few(const FewArgs &a, int w_type, cudaStream_t st) {
#define OOP_CASE(T) \
    case T: return launch_few<T>(a, st);
    switch (w_type) {
        OOP_CASE(OOP_TYPE_F32) OOP_CASE(OOP_TYPE_F16) OOP_CASE(OOP_TYPE_BF16) OOP_CASE(OOP_TYPE_Q4_0)
        OOP_CASE(OOP_TYPE_Q4_1) OOP_CASE(OOP_TYPE_Q5_0) OOP_CASE(OOP_TYPE_Q5_1) OOP_CASE(OOP_TYPE_Q8_0)
        OOP_CASE(OOP_TYPE_Q2_K) OOP_CASE(OOP_TYPE_Q3_K) OOP_CASE(OOP_TYPE_Q4_K) OOP_CASE(OOP_TYPE_Q5_K)
        OOP_CASE(OOP_TYPE_Q6_K)
    }
#undef OOP_CASE
    return cudaErrorInvalidValue;
}

// Rows of any type as P binary16 planes [P][rows][pitch] of a scaled value, hi + lo: a row
// is scaled by the power of two that brings its largest magnitude to 2^13 .. 2^14, so
// nothing overflows, what is above 2^-16 of the largest keeps 22 bits or more, and what is
// below is off by up to 2^-38 of the largest (half of binary16's smallest step, 2^-24, over
// 2^13).  That is relative to the row, not to a sum's terms: where the other matrix is zero
// under the largest, it shows in full.  factors: the inverse scales.  So two planes and three
// terms do for the forward products of f32; elsewhere, where sums run over other rows'
// scales, it takes three bfloat16 planes and six terms.  A warp takes a row, read once up to
// kHold * 256 columns; up to three matrices of the same columns in a launch.  512 tokens of
// f32 with kHold of 5, 10 and 20: K = 1280, F = 9728 94, 95 and 124 us, K = 2560 189, 165 and
// 182, K = 5120, F = 17408 681, 684 and 578: held rows cost registers, rows read twice
// bandwidth.
struct Scaled {
    const char *src;
    int64_t nb, rows;
    __half *dst;
    float *factors;
    int wide;
};
struct ScaledArgs {
    Scaled m[3];
    int count;
    int64_t cols, pitch;
};

template <int TYPE, int P>
__global__ void __launch_bounds__(256) halves_kernel(const __grid_constant__ ScaledArgs a) {
    constexpr int kHold = 10;
    let_next_start();
    const int lane = threadIdx.x & 31;
    int64_t r = blockIdx.x * 8LL + (threadIdx.x >> 5);
    int which = 0;
    while (which < a.count && r >= a.m[which].rows) r -= a.m[which++].rows;
    if (which == a.count) return;
    const Scaled &m = a.m[which];
    const char *row = m.src + r * m.nb;
    float held[kHold][8], top = 0.f;
    auto largest = [&](const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) top = v[i] == v[i] ? fmaxf(top, fabsf(v[i])) : __int_as_float(0x7f800000);
    };
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
        const int64_t c = (lane + 32 * h) * 8;
        if (c < a.cols) load8<TYPE>(row, c, a.cols, m.wide, held[h]);
    }
#pragma unroll
    for (int h = 0; h < kHold; ++h)
        if ((lane + 32 * h) * 8 < a.cols) largest(held[h]);
    for (int64_t c = (lane + 32 * kHold) * 8; c < a.cols; c += 32 * 8) {
        float v[8];
        load8<TYPE>(row, c, a.cols, m.wide, v);
        largest(v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // 13 - floor(log2 top), within a float's exponents; 0 for a row of zeros or one that is not
    // finite
    const int exponent = static_cast<int>(__float_as_uint(top) >> 23);
    const int e = top > 0.f && exponent < 255 ? max(-126, min(126, 13 + 127 - exponent)) : 0;
    const float scale = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    if (lane == 0) m.factors[r] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    __half *d = m.dst + r * a.pitch;
    const int64_t plane = m.rows * a.pitch;
    auto put = [&](const float (&v)[8], int64_t c) {
        float left[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) left[i] = v[i] * scale;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            __half h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[i] = __float2half_rn(left[i]);
                left[i] -= __half2float(h[i]);
            }
            uint4 w;
            __builtin_memcpy(&w, h, 16);
            *reinterpret_cast<uint4 *>(d + p * plane + c) = w;
        }
    };
#pragma unroll
    for (int h = 0; h < kHold; ++h)
        if ((lane + 32 * h) * 8 < a.cols) put(held[h], (lane + 32 * h) * 8);
    for (int64_t c = (lane + 32 * kHold) * 8; c < a.cols; c += 32 * 8) {
        float v[8];
        load8<TYPE>(row, c, a.cols, m.wide, v);
        put(v, c);
    }
}

cudaError_t launch_halves(const ScaledArgs &a, int type, cudaStream_t st) {
    int64_t rows = 0;
    for (int i = 0; i < a.count; ++i) rows += a.m[i].rows;
    const unsigned g = static_cast<unsigned>((rows + 7) / 8);
#define OOP_CASE(T, P) \
    case T: halves_kernel<T, P><<<g, 256, 0, st>>>(a); break;
    switch (type) {
        OOP_CASE(OOP_TYPE_F16, 1) OOP_CASE(OOP_TYPE_BF16, 1) OOP_CASE(OOP_TYPE_F32, 2) OOP_CASE(OOP_TYPE_Q4_0, 2)
        OOP_CASE(OOP_TYPE_Q4_1, 2) OOP_CASE(OOP_TYPE_Q5_0, 2) OOP_CASE(OOP_TYPE_Q5_1, 2) OOP_CASE(OOP_TYPE_Q8_0, 2)
        OOP_CASE(OOP_TYPE_Q2_K, 2) OOP_CASE(OOP_TYPE_Q3_K, 2) OOP_CASE(OOP_TYPE_Q4_K, 2) OOP_CASE(OOP_TYPE_Q5_K, 2)
        OOP_CASE(OOP_TYPE_Q6_K, 2)
    }
#undef OOP_CASE
    ++g_kernel_launches;
    return cudaGetLastError();
}

// dgate and dup as P planes [P][2][T][pitch]: dgate = dh up act'(gate), dup = dh act(gate).
template <int DTYPE, int TYPE, int P>
__global__ void __launch_bounds__(256) gate_back_kernel(const char *dh, int64_t nb_dh, const char *gate, const char *up, int64_t nb_gu,
                                                        __nv_bfloat16 *dst, int64_t pitch, int64_t F, int64_t T, int act, int wide) {
    const int64_t per_row = pitch / 8;
    let_next_start();
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < T * per_row; i += gridDim.x * 256LL) {
        const int64_t t = i / per_row, c = (i - t * per_row) * 8;
        float d[8], g[8], u[8];
        if (wide && c + 8 <= F) {
            Eight<DTYPE> ed;
            Eight<TYPE> eg, eu;
            ed.load(dh + t * nb_dh, c);
            eg.load(gate + t * nb_gu, c);
            eu.load(up + t * nb_gu, c);
            ed.get(d);
            eg.get(g);
            eu.get(u);
        } else {
            load8<DTYPE>(dh + t * nb_dh, c, F, 0, d);
            load8<TYPE>(gate + t * nb_gu, c, F, 0, g);
            load8<TYPE>(up + t * nb_gu, c, F, 0, u);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float slope;
            const float a = activation_and_slope(act, g[k], slope);
            g[k] = d[k] * u[k] * slope;
            u[k] = d[k] * a;
        }
        store_planes<P>(g, dst + t * pitch + c, 2 * T * pitch);
        store_planes<P>(u, dst + (T + t) * pitch + c, 2 * T * pitch);
    }
}

template <int DTYPE, int P>
void launch_gate_back(int x_type, const char *dh, int64_t nb_dh, const char *gate, const char *up, int64_t nb_gu, void *dst,
                      int64_t pitch, int64_t F, int64_t T, int act, int wide, cudaStream_t st) {
    auto *d = static_cast<__nv_bfloat16 *>(dst);
    const unsigned g = blocks_of(T * pitch / 8);
    if (x_type == OOP_TYPE_F32) gate_back_kernel<DTYPE, OOP_TYPE_F32, P><<<g, 256, 0, st>>>(dh, nb_dh, gate, up, nb_gu, d, pitch, F, T, act, wide);
    else if (x_type == OOP_TYPE_F16) gate_back_kernel<DTYPE, OOP_TYPE_F16, P><<<g, 256, 0, st>>>(dh, nb_dh, gate, up, nb_gu, d, pitch, F, T, act, wide);
    else gate_back_kernel<DTYPE, OOP_TYPE_BF16, P><<<g, 256, 0, st>>>(dh, nb_dh, gate, up, nb_gu, d, pitch, F, T, act, wide);
    ++g_kernel_launches;
}

// ---- operands -------------------------------------------------------------

// How a matrix of a type goes to the tensor cores: as it is (0: not even copied), or as so
// many 16-bit planes in the workspace.
struct Form {
    int planes;        // terms of a value
    bool half, copy;   // binary16; in the workspace
    bool scaled;       // by rows
};

// `native`: the other operand has this 16-bit type too.  `precise`: the product is wanted
// to 24 bits.
Form form_of(int type, bool native, bool precise, bool aligned) {
    if (native) return {1, type == OOP_TYPE_F16, !aligned, false};
    if (type == OOP_TYPE_BF16) return {1, false, !aligned, false};
    if (type == OOP_TYPE_F16) return {2, false, true, false};              // 11 bits: two planes hold them
    return {precise ? 3 : 2, false, true, false};
}

size_t form_bytes(const Form &f, int64_t cols, int64_t rows) {
    if (!f.copy) return 0;
    return pair::round256(static_cast<size_t>(f.planes) * static_cast<size_t>(rows * pair::round8(cols)) * 2) +
           (f.scaled ? pair::round256(static_cast<size_t>(rows) * 4) : 0);
}

struct ForwardForms {
    Form x, w;
};
ForwardForms forward_forms(int x_type, int w_type, bool aligned) {
    const bool native = x_type == w_type && x_type != OOP_TYPE_F32 && plain_size(x_type) == 2;
    if (x_type == OOP_TYPE_F32)                            // a sum's factors are of its row and its column: both can be scaled
        return {{2, true, true, true}, {plain_size(w_type) == 2 ? 1 : 2, true, true, true}};
    return {form_of(x_type, native, false, aligned), form_of(w_type, native, false, aligned)};
}
struct BackForms {
    Form d, x, w;
};
// dgate and dup of small calls keep 16 bits where dh has 8: with few tokens reading the
// weights takes longer than twice the products, in small products their launch does (2^31
// elements: 9 us), and a gradient of few terms would show their rounding.
BackForms back_forms(int dh_type, int x_type, int w_type, const int64_t ne[3], bool aligned) {
    const bool precise = dh_type == OOP_TYPE_F32;
    const double size = static_cast<double>(ne[0]) * static_cast<double>(ne[1]) * static_cast<double>(ne[2]);
    const bool small = ne[2] <= pair::kTileM || size <= 0x1p31;
    return {{precise ? 3 : small ? 2 : 1, false, true, false}, form_of(x_type, false, precise, aligned), form_of(w_type, false, precise, aligned)};
}

// A matrix {cols, rows} as an operand whose k (or rows) are contiguous: the caller's
// memory, or planes that this call writes at `at`, which moves on.
cudaError_t operand(const Form &f, const void *src, int type, int64_t nb, int64_t cols, int64_t rows, bool rows_contiguous,
                    char *&at, pair::Operand &o, cudaStream_t st) {
    o = {src, cols, rows, nb, 0, 1, rows_contiguous, f.half};
    if (!f.copy) return cudaSuccess;
    const int64_t pitch = pair::round8(cols);
    o.p = at;
    o.pitch_bytes = pitch * 2;
    o.matrix_bytes = rows * pitch * 2;
    o.matrices = f.planes;
    at += form_bytes(f, cols, rows);
    if (f.planes == 1) return launch_planes_of<0>(src, type, nb, cols, rows, const_cast<void *>(o.p), pitch, st);
    return f.planes == 2 ? launch_planes_of<2>(src, type, nb, cols, rows, const_cast<void *>(o.p), pitch, st)
                         : launch_planes_of<3>(src, type, nb, cols, rows, const_cast<void *>(o.p), pitch, st);
}

// The same for a matrix whose rows are scaled, k contiguous: what halves_kernel has to do.
Scaled scaled_operand(const Form &f, const void *src, int64_t nb, int64_t cols, int64_t rows, char *&at, pair::Operand &o) {
    const int64_t pitch = pair::round8(cols);
    o = {at, cols, rows, pitch * 2, rows * pitch * 2, f.planes, false, true};
    Scaled m = {static_cast<const char *>(src), nb, rows, reinterpret_cast<__half *>(at), nullptr, is_aligned(src, 16) && nb % 16 == 0};
    at += form_bytes(f, cols, rows);
    m.factors = reinterpret_cast<float *>(at - pair::round256(static_cast<size_t>(rows) * 4));
    return m;
}

// Tiles of 256 columns, or of 128 where those leave SMs idle: the time of the waves (a
// narrow tile reads A as often as a wide one for half the sums).
bool narrow_tiles(int64_t M, int64_t N, int64_t batches, int wide_cols) {
    auto waves = [&](int64_t cols) {
        const int64_t tiles = (M + pair::kTileM - 1) / pair::kTileM * ((N + cols - 1) / cols) * batches;
        return (tiles + pair::kPairs - 1) / pair::kPairs;
    };
    return waves(wide_cols / 2) * 23 < waves(wide_cols) * 40;
}

// A gradient's product: narrow tiles or wide ones, and which go in parts of k.  333 x 1001
// x 3074 in f32 has 16 tiles, whose 50 stages would take 40 us; 8192 x 2560 x 19456 fills
// four waves and a fifth of the next, which as parts takes a quarter of its time.
struct GradientPlan {
    bool narrow;
    pair::TileMap map;
    size_t slots;
};
GradientPlan gradient_plan(int64_t M, int64_t N, int64_t K, int planes_a, int planes_b, int64_t batches, int64_t segments) {
    GradientPlan p;
    const int64_t stages = (K + pair::kDepth - 1) / pair::kDepth * segments;
    p.narrow = narrow_tiles(M, N, batches, 256);
    const int64_t cols = p.narrow ? 128 : 256;
    p.map = pair::tile_map(M, N, cols, stages, pair::count_terms(planes_a, planes_b), batches, false, true);
    p.slots = pair::slot_bytes(p.map, batches, cols);
    return p;
}

// Sums of the parts to p0 (and p1: the second batch's).
template <int TYPE, int BN>
__global__ void __launch_bounds__(256) join_kernel(const pair::TileMap map, const float *slots, int64_t M, int64_t N, char *p0, char *p1,
                                                   int64_t nb) {
    let_next_start();
    wait_previous();
    pair::each_joined<BN>(map, slots, [&](int z, int64_t r, int64_t c, float4 v) {
        if (r >= M) return;
        auto *row = row_of<TYPE>(z ? p1 : p0, nb, r);
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < N) row[c + i] = from_float<TYPE>(f[i]);
    });
}

template <int TYPE, int BN>
cudaError_t launch_join(const pair::TileMap &m, const pair::Spec &s, cudaStream_t st) {
    ++g_kernel_launches;
    return launch_dependent(join_kernel<TYPE, BN>, dim3(static_cast<unsigned>(pair::kJoinCtas * pair::tiles_in_parts(m, s.batches))), 256, 0, st, m,
                            static_cast<const float *>(s.out.slots), s.M, s.N, static_cast<char *>(s.out.p0),
                            static_cast<char *>(s.out.p1), s.out.nb0);
}

template <bool FOLD>
cudaError_t gradient(pair::Spec s, void *slots, int *status, cudaStream_t st) {
    const GradientPlan p = gradient_plan(s.M, s.N, s.K, s.planes_a, s.planes_b, s.batches, s.segments);
    s.in_parts = true;
    s.out.slots = static_cast<float *>(slots);
    const cudaError_t e = p.narrow ? pair::launch<pair::kPlain, FOLD, 128>(s, status, st) : pair::launch<pair::kPlain, FOLD, 256>(s, status, st);
    if (e != cudaSuccess || p.map.parts == 1) return e;
    if (s.out.type == OOP_TYPE_F32)
        return p.narrow ? launch_join<OOP_TYPE_F32, 128>(p.map, s, st) : launch_join<OOP_TYPE_F32, 256>(p.map, s, st);
    return p.narrow ? launch_join<OOP_TYPE_BF16, 128>(p.map, s, st) : launch_join<OOP_TYPE_BF16, 256>(p.map, s, st);
}

cudaError_t zero_rows(void *p, int64_t nb, int64_t row_bytes, int64_t rows, cudaStream_t st) {
    if (rows == 0 || row_bytes == 0) return cudaSuccess;
    return cudaMemset2DAsync(p, static_cast<size_t>(rows > 1 ? nb : row_bytes), 0, static_cast<size_t>(row_bytes),
                             static_cast<size_t>(rows), st);
}

int check_ffn(int x_type, int w_type, const int64_t ne[3], int act) {
    if (!ne) return OOP_ERR_NULL;
    const int qk = type_block_elems(w_type);
    if (!plain_size(x_type) || qk < 0) return OOP_ERR_TYPE;
    for (int i = 0; i < 3; ++i)
        if (ne[i] < 0 || ne[i] > 0x7fffffffLL) return OOP_ERR_SHAPE;
    if (ne[0] % qk != 0) return OOP_ERR_SHAPE;
    for (int i = 0; i < 3; ++i) {
        const int rc = check_extent(ne[i], ne[(i + 1) % 3]);
        if (rc != OOP_OK) return rc;
    }
    if (act < OOP_ACT_SILU || act > OOP_ACT_RELU) return OOP_ERR_VALUE;
    return OOP_OK;
}

int64_t weight_row_bytes(int w_type, int64_t K) { return K / type_block_elems(w_type) * type_block_bytes(w_type); }

// The alignment that elements of an oop_type need, and the unit of their row stride.
int unit_of(int type) { return type == OOP_TYPE_F32 ? 4 : 2; }

int check_weights(const void *wg, const void *wu, int w_type, int64_t nb_w, int64_t K, int64_t F) {
    int rc = check_row_stride(weight_row_bytes(w_type, K), F, nb_w, unit_of(w_type), false);
    if (rc == OOP_OK && K > 0 && F > 0) rc = check_pointer(wg, unit_of(w_type));
    if (rc == OOP_OK && K > 0 && F > 0) rc = check_pointer(wu, unit_of(w_type));
    return rc;
}

// Rows that 16-byte accesses can take as they are, and those that TMA can: apart as well.
bool rows_aligned(const void *p, int64_t nb, int64_t rows) { return is_aligned(p, 16) && (rows <= 1 || nb % 16 == 0); }
bool rows_apart(const void *p, int64_t nb, int64_t rows, int64_t row_bytes) {
    return rows_aligned(p, nb, rows) && (rows <= 1 || nb >= row_bytes);
}

int check_workspace(const void *ws, size_t have, size_t need) {
    return need == 0 || (ws && have >= need && is_aligned(ws, 256)) ? OOP_OK : OOP_ERR_WORKSPACE;
}

}  // namespace
}  // namespace oop

using namespace oop;

extern "C" {

size_t oop_gated_ffn_workspace_size(int x_type, int w_type, const int64_t ne[3], int aligned) {
    if (check_ffn(x_type, w_type, ne, 0) != OOP_OK || few_tokens(ne[2], ne[0], x_type, w_type)) return 0;
    const ForwardForms f = forward_forms(x_type, w_type, aligned != 0);
    return form_bytes(f.x, ne[0], ne[2]) + 2 * form_bytes(f.w, ne[0], ne[1]);
}

size_t oop_gated_ffn_back_workspace_size(int dh_type, int x_type, int w_type, const int64_t ne[3], int aligned) {
    if (!gradient_type(dh_type) || check_ffn(x_type, w_type, ne, 0) != OOP_OK) return 0;
    const BackForms f = back_forms(dh_type, x_type, w_type, ne, aligned != 0);
    const int64_t K = ne[0], F = ne[1], T = ne[2];
    // the parts of the two products follow each other in one place
    const size_t parts = std::max(gradient_plan(T, K, F, f.d.planes, f.w.planes, 1, 2).slots,
                                  gradient_plan(F, K, T, f.d.planes, f.x.planes, 2, 1).slots);
    return form_bytes(f.d, F, 2 * T) + form_bytes(f.x, K, T) + 2 * form_bytes(f.w, K, F) + parts;
}

int oop_gated_ffn(const void *x, int x_type, int64_t nb_x, const void *w_gate, const void *w_up, int w_type,
                  int64_t nb_w, void *h, int64_t nb_h, void *gate, void *up, int64_t nb_gu, const int64_t ne[3],
                  int act, void *workspace, size_t workspace_bytes, void *stream) {
    g_kernel_launches = 0;
    int rc = check_ffn(x_type, w_type, ne, act);
    if (rc != OOP_OK) return rc;
    const int64_t K = ne[0], F = ne[1], T = ne[2];
    const int size = plain_size(x_type);
    if ((rc = check_row_stride(K * size, T, nb_x, size, false)) != OOP_OK) return rc;
    if ((rc = check_row_stride(F * size, T, nb_h, size, true)) != OOP_OK) return rc;
    if ((gate == nullptr) != (up == nullptr)) return OOP_ERR_NULL;
    if (gate && (rc = check_row_stride(F * size, T, nb_gu, size, true)) != OOP_OK) return rc;
    if ((rc = check_weights(w_gate, w_up, w_type, nb_w, K, T ? F : 0)) != OOP_OK) return rc;
    if (T == 0 || F == 0) return OOP_OK;
    if (K > 0 && (rc = check_pointer(x, size)) != OOP_OK) return rc;
    if ((rc = check_pointer(h, size)) != OOP_OK) return rc;
    if (gate && ((rc = check_pointer(gate, size)) != OOP_OK || (rc = check_pointer(up, size)) != OOP_OK)) return rc;
    const int64_t w_bytes = weight_row_bytes(w_type, K);
    const bool aligned = rows_apart(x, nb_x, T, K * size) && rows_apart(w_gate, nb_w, F, w_bytes) && rows_apart(w_up, nb_w, F, w_bytes);
    if ((rc = check_workspace(workspace, workspace_bytes, oop_gated_ffn_workspace_size(x_type, w_type, ne, aligned))) != OOP_OK)
        return rc;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (K == 0) {                                          // sums of nothing: act(0) * 0
        cudaError_t e = zero_rows(h, nb_h, F * size, T, st);
        if (gate && e == cudaSuccess) e = zero_rows(gate, nb_gu, F * size, T, st);
        if (gate && e == cudaSuccess) e = zero_rows(up, nb_gu, F * size, T, st);
        return cuda_status(e);
    }
    if (few_tokens(T, K, x_type, w_type)) {
        FewArgs a = {static_cast<const char *>(x), {static_cast<const char *>(w_gate), static_cast<const char *>(w_up)},
                     static_cast<char *>(h), static_cast<char *>(gate), static_cast<char *>(up), nb_x, nb_w, nb_h, nb_gu, K, F,
                     static_cast<int>(T), x_type, act, 0};
        a.wide = rows_aligned(w_gate, nb_w, F) && rows_aligned(w_up, nb_w, F);
        return cuda_status(launch_few(a, w_type, st));
    }
    const ForwardForms f = forward_forms(x_type, w_type, aligned);
    char *at = static_cast<char *>(workspace);
    pair::Spec s = {};
    cudaError_t e = cudaSuccess;
    if (f.x.scaled) {
        ScaledArgs a = {};
        a.cols = K, a.pitch = pair::round8(K);
        a.m[a.count++] = scaled_operand(f.x, x, nb_x, K, T, at, s.a);
        s.out.row_scale = a.m[0].factors;
        if (w_type != OOP_TYPE_F32) {                      // another type: a launch of its own
            e = launch_halves(a, x_type, st);
            a.count = 0;
        }
        const void *w[2] = {w_gate, w_up};
        for (int i = 0; i < 2; ++i) {
            a.m[a.count] = scaled_operand(f.w, w[i], nb_w, K, F, at, s.b[i]);
            s.out.col_scale[i] = a.m[a.count++].factors;
        }
        if (e == cudaSuccess) e = launch_halves(a, w_type, st);
    } else {
        e = operand(f.x, x, x_type, nb_x, K, T, false, at, s.a, st);
        if (e == cudaSuccess) e = operand(f.w, w_gate, w_type, nb_w, K, F, false, at, s.b[0], st);
        if (e == cudaSuccess) e = operand(f.w, w_up, w_type, nb_w, K, F, false, at, s.b[1], st);
    }
    if (e != cudaSuccess) return cuda_status(e);
    s.M = T, s.N = F, s.K = K;
    s.batches = s.segments = 1;
    s.planes_a = f.x.planes, s.planes_b = f.w.planes;
    s.a_plane = s.b_plane = 1;
    s.out.p0 = h, s.out.p1 = gate, s.out.p2 = up;
    s.out.nb0 = nb_h, s.out.nb1 = nb_gu;
    s.out.type = x_type, s.out.act = act;
    s.out.wide = F * size % 16 == 0 && rows_aligned(h, nb_h, T) &&
                 (!gate || (rows_aligned(gate, nb_gu, T) && rows_aligned(up, nb_gu, T)));
    const bool narrow = narrow_tiles(T, F, 1, 128);
    if (x_type == OOP_TYPE_F32) e = narrow ? pair::launch<pair::kGate, true, 128>(s, status, st) : pair::launch<pair::kGate, true, 256>(s, status, st);
    else e = narrow ? pair::launch<pair::kGate, false, 128>(s, status, st) : pair::launch<pair::kGate, false, 256>(s, status, st);
    return cuda_status(e);
}

int oop_gated_ffn_back(const void *dh, int dh_type, int64_t nb_dh, const void *x, int x_type, int64_t nb_x,
                       const void *w_gate, const void *w_up, int w_type, int64_t nb_w, const void *gate,
                       const void *up, int64_t nb_gu, void *dx, int64_t nb_dx, void *dw_gate, void *dw_up,
                       int64_t nb_dw, const int64_t ne[3], int act, void *workspace, size_t workspace_bytes,
                       void *stream) {
    g_kernel_launches = 0;
    int rc = check_ffn(x_type, w_type, ne, act);
    if (rc != OOP_OK) return rc;
    if (!gradient_type(dh_type)) return OOP_ERR_TYPE;
    const int64_t K = ne[0], F = ne[1], T = ne[2];
    const int size = plain_size(x_type), d_size = plain_size(dh_type);
    if ((dw_gate == nullptr) != (dw_up == nullptr)) return OOP_ERR_NULL;
    if ((rc = check_row_stride(F * d_size, T, nb_dh, d_size, false)) != OOP_OK) return rc;
    if ((rc = check_row_stride(K * size, T, nb_x, size, false)) != OOP_OK) return rc;
    if ((rc = check_row_stride(F * size, T, nb_gu, size, false)) != OOP_OK) return rc;
    if (dx && (rc = check_row_stride(K * d_size, T, nb_dx, d_size, true)) != OOP_OK) return rc;
    if (dw_gate && (rc = check_row_stride(K * d_size, F, nb_dw, d_size, true)) != OOP_OK) return rc;
    if ((rc = check_weights(w_gate, w_up, w_type, nb_w, K, dx && T ? F : 0)) != OOP_OK) return rc;
    const bool want_dx = dx && T > 0 && K > 0, want_dw = dw_gate && F > 0 && K > 0;
    if (!want_dx && !want_dw) return OOP_OK;
    if (T > 0 && F > 0) {
        if ((rc = check_pointer(dh, d_size)) != OOP_OK) return rc;
        if ((rc = check_pointer(gate, size)) != OOP_OK) return rc;
        if ((rc = check_pointer(up, size)) != OOP_OK) return rc;
        if (want_dw && (rc = check_pointer(x, size)) != OOP_OK) return rc;
    }
    if (want_dx && (rc = check_pointer(dx, d_size)) != OOP_OK) return rc;
    if (want_dw && ((rc = check_pointer(dw_gate, d_size)) != OOP_OK || (rc = check_pointer(dw_up, d_size)) != OOP_OK)) return rc;
    const int64_t w_bytes = weight_row_bytes(w_type, K);
    const bool aligned = rows_apart(x, nb_x, T, K * size) && rows_apart(w_gate, nb_w, F, w_bytes) && rows_apart(w_up, nb_w, F, w_bytes);
    if ((rc = check_workspace(workspace, workspace_bytes, oop_gated_ffn_back_workspace_size(dh_type, x_type, w_type, ne, aligned))) != OOP_OK)
        return rc;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (T == 0 || F == 0) {                                // sums of nothing
        if (want_dx) e = zero_rows(dx, nb_dx, K * d_size, T, st);
        if (want_dw && e == cudaSuccess) e = zero_rows(dw_gate, nb_dw, K * d_size, F, st);
        if (want_dw && e == cudaSuccess) e = zero_rows(dw_up, nb_dw, K * d_size, F, st);
        return cuda_status(e);
    }
    const BackForms f = back_forms(dh_type, x_type, w_type, ne, aligned);
    char *at = static_cast<char *>(workspace);
    const int64_t pitch = pair::round8(F);
    // [plane][gate, up][T][pitch]
    pair::Operand d = {at, F, T, pitch * 2, T * pitch * 2, 2 * f.d.planes, false, false};
    const int wide = rows_aligned(dh, nb_dh, T) && rows_aligned(gate, nb_gu, T) && rows_aligned(up, nb_gu, T);
    const char *dp = static_cast<const char *>(dh), *gp = static_cast<const char *>(gate), *up_ = static_cast<const char *>(up);
    if (dh_type == OOP_TYPE_F32) launch_gate_back<OOP_TYPE_F32, 3>(x_type, dp, nb_dh, gp, up_, nb_gu, at, pitch, F, T, act, wide, st);
    else if (f.d.planes == 2) launch_gate_back<OOP_TYPE_BF16, 2>(x_type, dp, nb_dh, gp, up_, nb_gu, at, pitch, F, T, act, wide, st);
    else launch_gate_back<OOP_TYPE_BF16, 1>(x_type, dp, nb_dh, gp, up_, nb_gu, at, pitch, F, T, act, wide, st);
    e = cudaGetLastError();
    at += form_bytes(f.d, F, 2 * T);
    char *parts = at + form_bytes(f.x, K, T) + 2 * form_bytes(f.w, K, F);
    auto run = [&](const pair::Spec &s) {
        return dh_type == OOP_TYPE_F32 ? gradient<true>(s, parts, status, st) : gradient<false>(s, parts, status, st);
    };
    if (want_dx && e == cudaSuccess) {                     // [dgate dup] [Wg; Wu]: two segments of F
        pair::Spec s = {};
        s.a = d;
        e = operand(f.w, w_gate, w_type, nb_w, K, F, true, at, s.b[0], st);
        if (e == cudaSuccess) e = operand(f.w, w_up, w_type, nb_w, K, F, true, at, s.b[1], st);
        s.M = T, s.N = K, s.K = F;
        s.batches = 1, s.segments = 2;
        s.planes_a = f.d.planes, s.planes_b = f.w.planes;
        s.a_plane = 2, s.a_seg = 1, s.b_plane = 1;
        s.out.p0 = dx, s.out.nb0 = nb_dx, s.out.type = dh_type, s.out.alpha = s.out.beta = 1.f;
        s.out.wide = K * d_size % 16 == 0 && rows_aligned(dx, nb_dx, T);
        if (e == cudaSuccess) e = run(s);
    }
    if (want_dw && e == cudaSuccess) {                     // dgate' x and dup' x: two batches
        pair::Spec s = {};
        s.a = d;
        s.a.rows_contiguous = true;
        e = operand(f.x, x, x_type, nb_x, K, T, true, at, s.b[0], st);
        s.b[1] = s.b[0];
        s.M = F, s.N = K, s.K = T;
        s.batches = 2, s.segments = 1;
        s.planes_a = f.d.planes, s.planes_b = f.x.planes;
        s.a_plane = 2, s.a_batch = 1, s.b_plane = 1;
        s.out.p0 = dw_gate, s.out.p1 = dw_up, s.out.nb0 = nb_dw, s.out.type = dh_type, s.out.alpha = s.out.beta = 1.f;
        s.out.wide = K * d_size % 16 == 0 && rows_aligned(dw_gate, nb_dw, F) && rows_aligned(dw_up, nb_dw, F);
        if (e == cudaSuccess) e = run(s);
    }
    return cuda_status(e);
}

}  // extern "C"
