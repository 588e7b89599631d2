// qk_norm_rope.cu -- RMS norm of every query and key head and the rotation by the token's
// position, in one pass, and its backward pass.
//
//   r = (sum_d x^2 / D + eps)^(-1/2),  n = x r w,  y = R(pos) n
//   dn = R(-pos) dy,  g = dn w,  dx = r (g - x r^2 sum_d (g x) / D),
//   dw = sum over tokens and heads of dn x r
//
// Bound by memory: x is read once and y written once, nothing else is of their size.
// bf16, 16384 tokens of 32 + 8 heads of 128: 62 us, 5.4 TB/s (80% of the measured copy
// rate), backward 108 us, 4.6 TB/s (69%): half of the issue slots are taken, and 16 warps
// per SM wait for their loads and shuffles.  A head is held by a group of 2, 4 .. 32
// lanes.  A lane's unit is two chunks of E elements that hold whole pairs: chunk j of the
// first half of the rotated elements and its partner in the second half, or two
// neighbouring chunks.  So a rotation needs no other lane, and a lane's frequencies and
// weights are the same for every head: they stay in registers.
//
// The angle pos * freq is held in turns as a 64-bit fraction: freq / 2 pi is rounded once
// to 2^-64 turns, and the product with the integer position wraps around as the angle
// does, so no position loses precision.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "oop_internal.cuh"
#include "rows.cuh"

namespace oop {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxHead = 1024;

// The heads of the queries or of the keys, for either direction.
struct Side {
    const void *x, *dy, *w;
    void *out;                       // y, or dx
    int64_t x_head, x_tok, dy_head, dy_tok, out_head, out_tok;   // byte strides
    float *partial;                  // one row of D sums for each CTA of this side, or NULL
    int heads, ctas;
    int splits;                      // warps that share a token's heads
};

struct Args {
    Side side[2];
    const int32_t *pos;
    const float *freqs;
    int64_t T;
    int D, half, interleaved, group_shift, units, w_type;
    float eps, inv_d;
    float low;                       // sums of squares below it are taken again
};

// freq / (2 pi) modulo 1 as a 64-bit fraction: the 24-bit significand times 128 bits of 1
// / (2 pi), shifted by the exponent, in integers (64-bit floating point has a sixtieth of
// the rate here).  Exact to 2^-64 for |freq| < 2^40.
__device__ __forceinline__ uint64_t turns_of(float freq) {
    constexpr uint64_t kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;   // 2^128 / (2 pi)
    const uint32_t bits = __float_as_uint(freq);
    const int exponent = static_cast<int>(bits >> 23 & 0xffu);
    const uint64_t m = (bits & 0x7fffffu) | (exponent ? 0x800000u : 0u);
    const int shift = 64 + 150 - (exponent ? exponent : 1);        // freq = m 2^(64 - shift)
    const uint64_t low = m * kLo, carry = __umul64hi(m, kLo);
    const uint64_t mid = m * kHi + carry, top = __umul64hi(m, kHi) + (mid < carry);
    uint64_t v = 0;
    if (shift >= 128) v = shift < 192 ? top >> (shift - 128) : 0;
    else if (shift > 64) v = mid >> (shift - 64) | top << (128 - shift);
    else if (shift == 64) v = mid;
    else if (shift > 0) v = low >> shift | mid << (64 - shift);
    return bits >> 31 ? ~v + 1 : v;
}

__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    const float x = a * c - b * s;
    b = a * s + b * c;
    a = x;
}

// The turns per position of every pair, one copy for the CTA.
struct Steps {
    uint64_t of[kMaxHead / 2];
    float bad[kMaxHead / 2];         // NaN for a frequency that is not finite, else 0
    int any_bad;
};

__device__ __forceinline__ void fill_steps(Steps &s, const Args &a) {
    if (threadIdx.x == 0) s.any_bad = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.half; i += kThreads) {
        const float f = a.freqs[i], bad = f * 0.f;
        s.of[i] = bad == 0.f ? turns_of(f) : 0;
        s.bad[i] = bad;
        if (bad != 0.f) s.any_bad = 1;
    }
    __syncthreads();
}

// What a lane holds of one head: U units of two chunks.
template <int E, int U>
struct Lane {
    int c0[U], c1[U];                // first elements of the chunks; -1: none
    int freq[U];                     // first frequency; -1: not rotated

    __device__ __forceinline__ void place(const Args &a, int lane) {
        const int g = 1 << a.group_shift, rot_units = a.half / E;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = lane + u * g;
            c0[u] = c1[u] = freq[u] = -1;
            if (j >= a.units) continue;
            if (j < rot_units) {
                c0[u] = a.interleaved ? 2 * E * j : E * j;
                c1[u] = a.interleaved ? c0[u] + E : a.half + E * j;
                freq[u] = E * j;
            } else {
                c0[u] = 2 * a.half + 2 * E * (j - rot_units);
                c1[u] = c0[u] + E < a.D ? c0[u] + E : -1;        // E = 1 and an odd rest
            }
        }
    }
};

template <int E, int U>
struct Values {
    float a[U][E], b[U][E];
};

// A head as it lies in memory.
template <int TYPE, int E, int U>
struct Raw {
    Packed<TYPE, E> a[U], b[U];

    __device__ __forceinline__ void load(const char *row, bool exists, const Lane<E, U> &l) {
        using S = typename Plain<TYPE>::S;
        const S *p = reinterpret_cast<const S *>(row);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[u].raw = b[u].raw = {};
            if (exists && l.c0[u] >= 0) a[u] = load_stream<TYPE, E>(p + l.c0[u]);
            if (exists && l.c1[u] >= 0) b[u] = load_stream<TYPE, E>(p + l.c1[u]);
        }
    }
    __device__ __forceinline__ void get(Values<E, U> &v) const {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[u].get(v.a[u]);
            b[u].get(v.b[u]);
        }
    }
};

template <int TYPE, int E, int U>
__device__ __forceinline__ void store_head(char *row, const Values<E, U> &v, const Lane<E, U> &l) {
    using S = typename Plain<TYPE>::S;
    S *p = reinterpret_cast<S *>(row);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (l.c0[u] >= 0) store_stream<TYPE, E>(p + l.c0[u], v.a[u]);
        if (l.c1[u] >= 0) store_stream<TYPE, E>(p + l.c1[u], v.b[u]);
    }
}

// cos and sin of the token's angles; 0 turns for what is not rotated.  FAST: for results
// of 16 bits, the hardware's functions, off by 2^-21 on (-pi, pi).
template <bool FAST, int E, int U>
__device__ __forceinline__ void angles(float (&c)[U][E], float (&s)[U][E], int64_t pos,
                                       const Steps &steps, const Lane<E, U> &l) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int p = 0; p < E; ++p) {
            c[u][p] = 1.f;
            s[u][p] = 0.f;
            if (l.freq[u] < 0) continue;
            const uint64_t t = static_cast<uint64_t>(pos) * steps.of[l.freq[u] + p];
            const float half_turns = static_cast<float>(static_cast<int32_t>(t >> 32));
            if constexpr (FAST) {
                c[u][p] = __cosf(half_turns * (3.14159265f * 0x1p-31f));
                s[u][p] = __sinf(half_turns * (3.14159265f * 0x1p-31f));
            } else {
                sincospif(half_turns * 0x1p-31f, &s[u][p], &c[u][p]);
            }
            if (steps.any_bad) {
                s[u][p] += steps.bad[l.freq[u] + p];
                c[u][p] += steps.bad[l.freq[u] + p];
            }
        }
}

// The lane's pairs turned; DIR = -1: back.  Without INF what is not rotated is turned by 0:
// nothing in it may be Inf.
template <int DIR, bool INF, int E, int U>
__device__ __forceinline__ void rotate(Values<E, U> &v, const float (&c)[U][E], const float (&s)[U][E],
                                       bool interleaved, const Lane<E, U> &l) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (INF && l.freq[u] < 0) continue;
        if (E == 1 || !interleaved) {
#pragma unroll
            for (int p = 0; p < E; ++p) turn(v.a[u][p], v.b[u][p], c[u][p], DIR * s[u][p]);
        } else {
#pragma unroll
            for (int p = 0; p < E / 2; ++p) {
                turn(v.a[u][2 * p], v.a[u][2 * p + 1], c[u][p], DIR * s[u][p]);
                turn(v.b[u][2 * p], v.b[u][2 * p + 1], c[u][E / 2 + p], DIR * s[u][E / 2 + p]);
            }
        }
    }
}

__device__ __forceinline__ float sum_in_group(float v, int group, unsigned lanes) {
    for (int o = group >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(lanes, v, o);
    return v;
}
__device__ __forceinline__ float group_sum(float v, int group) { return sum_in_group(v, group, 0xffffffffu); }

template <int E, int U>
__device__ __forceinline__ float dot(const Values<E, U> &v, const Values<E, U> &w) {
    float s = 0.f, z = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            s = fmaf(v.a[u][i], w.a[u][i], s);
            z = fmaf(v.b[u][i], w.b[u][i], z);
        }
    return s + z;
}

// A head whose sum of squares has left fp32's range, or lost its bits below it.  Such heads
// are rare: their loops leave them out and take them again, by themselves, where the sum is
// that of the head times a power of two.
__device__ __forceinline__ bool out_of_range(float sum, const Args &a) {
    return !(sum >= a.low && sum < __int_as_float(0x7f800000));
}

__device__ __forceinline__ unsigned lanes_of_group(int group) {
    return (0xffffffffu >> (32 - group)) << (threadIdx.x & 31 & ~(group - 1));
}

// r of such a head, which keeps the power of two that `scale` returns (r is that of the
// scaled head).  One that is not finite, or 0 with eps = 0, stays as it is.  All lanes of a
// group come here together.
template <int E, int U>
__device__ __forceinline__ float rescaled(Values<E, U> &v, const Args &a, float &scale) {
    const int group = 1 << a.group_shift;
    const unsigned lanes = lanes_of_group(group);
    float top = sqrtf(a.eps);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) top = fmaxf(top, fmaxf(fabsf(v.a[u][i]), fabsf(v.b[u][i])));
    for (int o = group >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(lanes, top, o));
    const int exponent = static_cast<int>(__float_as_uint(top) >> 23);
    scale = top == 0.f || exponent == 255 ? 1.f : __uint_as_float(static_cast<uint32_t>(max(1, 254 - exponent)) << 23);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            v.a[u][i] *= scale;
            v.b[u][i] *= scale;
        }
    return rsqrtf(sum_in_group(dot(v, v), group, lanes) * a.inv_d + a.eps * scale * scale);
}

// Weights of both sides in shared memory, as floats.
__device__ __forceinline__ void fill_weights(float *w, const Side &s, int type, int D) {
    for (int i = threadIdx.x; i < D; i += kThreads) w[i] = s.w && s.heads ? load_any(s.w, type, i) : 1.f;
}

// A warp takes whole tokens, or with few tokens a share of a token's heads: the queries'
// and then the keys', its groups the heads in turn, kAhead turns' loads before the first
// is used.
template <int TYPE, int E, int U>
__global__ void __launch_bounds__(kThreads, U == 1 ? 2 : 1) forward_kernel(const __grid_constant__ Args a) {
    constexpr int kAhead = E * U <= 8 ? 4 : 1;
    __shared__ Steps steps;
    __shared__ __align__(16) float weights[2][kMaxHead];
    const int lane = threadIdx.x & 31, group = 1 << a.group_shift;
    const int groups = 32 >> a.group_shift, mine = lane >> a.group_shift;
    fill_weights(weights[0], a.side[0], a.w_type, a.D);
    fill_weights(weights[1], a.side[1], a.w_type, a.D);
    fill_steps(steps, a);
    Lane<E, U> l;
    l.place(a, lane & (group - 1));
    const int splits = a.side[0].splits, step = groups * splits;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); item < a.T * splits; item += warps) {
        const int64_t t = item / splits;
        const int share = static_cast<int>(item - t * splits);
        float c[U][E], sn[U][E];
        bool turned = false;
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            const Side &s = a.side[which];
            const char *x = static_cast<const char *>(s.x) + t * s.x_tok;
            char *y = static_cast<char *>(s.out) + t * s.out_tok;
            const float *w = weights[which];
#pragma unroll 1
            for (int h0 = share * groups; h0 < s.heads; h0 += step * kAhead) {
                Raw<TYPE, E, U> raw[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int h = h0 + k * step + mine;
                    raw[k].load(x + h * s.x_head, h < s.heads, l);
                }
                if (!turned) angles<TYPE != OOP_TYPE_F32>(c, sn, a.half ? a.pos[t] : 0, steps, l);
                turned = true;
                Values<E, U> wv;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        wv.a[u][i] = l.c0[u] < 0 ? 0.f : w[l.c0[u] + i];
                        wv.b[u][i] = l.c1[u] < 0 ? 0.f : w[l.c1[u] + i];
                    }
                auto finish = [&](auto inf, Values<E, U> &v, float r, int h, bool stored) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int i = 0; i < E; ++i) {
                            v.a[u][i] *= r * wv.a[u][i];
                            v.b[u][i] *= r * wv.b[u][i];
                        }
                    rotate<1, inf>(v, c, sn, a.interleaved, l);
                    if (stored) store_head<TYPE>(y + h * s.out_head, v, l);
                };
                unsigned again = 0;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    if (h0 + k * step >= s.heads) break;   // the same for the warp
                    const int h = h0 + k * step + mine;
                    Values<E, U> v;
                    raw[k].get(v);
                    const float sum = group_sum(dot(v, v), group);
                    const bool out = out_of_range(sum, a);
                    again |= out ? 1u << k : 0u;
                    finish(std::false_type(), v, rsqrtf(sum * a.inv_d + a.eps), h, h < s.heads && !out);
                }
                if (!__any_sync(0xffffffffu, again)) continue;
#pragma unroll 1
                for (int k = 0; k < kAhead; ++k) {
                    const int h = h0 + k * step + mine;
                    if (!(again >> k & 1) || h >= s.heads) continue;       // the same for the group
                    Raw<TYPE, E, U> one;
                    Values<E, U> v;
                    float scale;
                    one.load(x + h * s.x_head, true, l);   // not stored to yet, if y is x
                    one.get(v);
                    const float r = rescaled(v, a, scale);
                    finish(std::true_type(), v, r, h, true);
                }
            }
        }
    }
}

template <int DTYPE, int TYPE, int E, int U>
__global__ void __launch_bounds__(kThreads, U == 1 ? 2 : 1) backward_kernel(const __grid_constant__ Args a) {
    constexpr int kAhead = E * U <= 4 ? 4 : E * U <= 8 ? 2 : 1;
    __shared__ Steps steps;
    __shared__ __align__(16) float weights[kMaxHead];
    __shared__ int again[kThreads / 32];                   // a warp has left out heads
    if (threadIdx.x < kThreads / 32) again[threadIdx.x] = 0;           // before the barriers below
    const int which = blockIdx.x >= static_cast<unsigned>(a.side[0].ctas);
    const Side &s = a.side[which];
    const int lane = threadIdx.x & 31, group = 1 << a.group_shift;
    const int groups = 32 >> a.group_shift, mine = lane >> a.group_shift;
    fill_weights(weights, s, a.w_type, a.D);
    fill_steps(steps, a);
    Lane<E, U> l;
    l.place(a, lane & (group - 1));
    Values<E, U> dw = {};
    const int64_t cta = static_cast<int64_t>(blockIdx.x) - (which ? a.side[0].ctas : 0);
    const int64_t warps = static_cast<int64_t>(s.ctas) * (kThreads / 32);
    const int64_t first = cta * (kThreads / 32) + (threadIdx.x >> 5);
    const int step = groups * s.splits;
    float c[U][E], sn[U][E];
    auto weigh = [&](auto inf, Values<E, U> &x, Values<E, U> &d, float r) {        // x becomes x r, d becomes g
        rotate<-1, inf>(d, c, sn, a.interleaved, l);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < E; ++i) {
                x.a[u][i] *= r;
                x.b[u][i] *= r;
                dw.a[u][i] = fmaf(d.a[u][i], x.a[u][i], dw.a[u][i]);
                dw.b[u][i] = fmaf(d.b[u][i], x.b[u][i], dw.b[u][i]);
                d.a[u][i] *= l.c0[u] < 0 ? 0.f : weights[l.c0[u] + i];
                d.b[u][i] *= l.c1[u] < 0 ? 0.f : weights[l.c1[u] + i];
            }
    };
    auto finish = [&](const Values<E, U> &x, Values<E, U> &d, float r, float m) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < E; ++i) {
                d.a[u][i] = r * (d.a[u][i] - x.a[u][i] * m);
                d.b[u][i] = r * (d.b[u][i] - x.b[u][i] * m);
            }
    };
    for (int64_t item = first; item < a.T * s.splits; item += warps) {
        const int64_t t = item / s.splits;
        const int share = static_cast<int>(item - t * s.splits);
        const char *xt = static_cast<const char *>(s.x) + t * s.x_tok, *dt = static_cast<const char *>(s.dy) + t * s.dy_tok;
        char *yt = static_cast<char *>(s.out) + t * s.out_tok;
        for (int h0 = share * groups; h0 < s.heads; h0 += step * kAhead) {
            Raw<TYPE, E, U> raw_x[kAhead];
            Raw<DTYPE, E, U> raw_d[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {             // what does not exist is 0, and adds nothing
                const int h = h0 + k * step + mine;
                raw_x[k].load(xt + h * s.x_head, h < s.heads, l);
                raw_d[k].load(dt + h * s.dy_head, h < s.heads, l);
            }
            if (h0 == share * groups) angles<DTYPE != OOP_TYPE_F32>(c, sn, a.half ? a.pos[t] : 0, steps, l);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (h0 + k * step >= s.heads) break;
                const int h = h0 + k * step + mine;
                Values<E, U> x, d;
                raw_x[k].get(x);
                raw_d[k].get(d);
                const float sum = group_sum(dot(x, x), group);
                const bool out = out_of_range(sum, a);
                if (out) again[threadIdx.x >> 5] = 1;      // in shared memory: the registers are all taken
                float r = rsqrtf(sum * a.inv_d + a.eps);
                if (h >= s.heads || out) r = 0.f;          // adds nothing; eps = 0: not 0 * Inf
                weigh(std::false_type(), x, d, r);
                finish(x, d, r, group_sum(dot(d, x), group) * a.inv_d);
                if (h < s.heads && !out) store_head<DTYPE>(yt + h * s.out_head, d, l);
            }
        }
    }
    __syncwarp();
    if (again[threadIdx.x >> 5]) {                         // those left out, in a loop of their own for the same reason
#pragma unroll 1
        for (int64_t item = first; item < a.T * s.splits; item += warps) {
            const int64_t t = item / s.splits;
            const int share = static_cast<int>(item - t * s.splits);
            angles<DTYPE != OOP_TYPE_F32>(c, sn, a.half ? a.pos[t] : 0, steps, l);
#pragma unroll 1
            for (int h0 = share * groups; h0 < s.heads; h0 += step) {
                const int h = h0 + mine;
                Raw<TYPE, E, U> raw_x;
                Raw<DTYPE, E, U> raw_d;
                Values<E, U> x, d;
                raw_x.load(static_cast<const char *>(s.x) + t * s.x_tok + h * s.x_head, h < s.heads, l);
                raw_x.get(x);
                if (!out_of_range(group_sum(dot(x, x), group), a) || h >= s.heads) continue;       // the same for the group
                raw_d.load(static_cast<const char *>(s.dy) + t * s.dy_tok + h * s.dy_head, true, l);       // not stored to, if dx is dy
                raw_d.get(d);
                float scale;
                const float r = rescaled(x, a, scale);
                weigh(std::true_type(), x, d, r);
                finish(x, d, r, sum_in_group(dot(d, x), group, lanes_of_group(group)) * a.inv_d);
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        d.a[u][i] *= scale;
                        d.b[u][i] *= scale;
                    }
                store_head<DTYPE>(static_cast<char *>(s.out) + t * s.out_tok + h * s.out_head, d, l);
            }
        }
    }
    if (!s.partial) return;
    // the CTA's sums: those of a warp's groups, then the warps' in their order
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i)
            for (int o = group; o < 32; o <<= 1) {
                dw.a[u][i] += __shfl_xor_sync(0xffffffffu, dw.a[u][i], o);
                dw.b[u][i] += __shfl_xor_sync(0xffffffffu, dw.b[u][i], o);
            }
    float *part = weights;                                 // no longer needed
    for (int turn_of = 0; turn_of < kThreads / 32; ++turn_of) {
        __syncthreads();
        if (static_cast<int>(threadIdx.x >> 5) != turn_of || mine != 0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (l.c0[u] >= 0) part[l.c0[u] + i] = (turn_of ? part[l.c0[u] + i] : 0.f) + dw.a[u][i];
                if (l.c1[u] >= 0) part[l.c1[u] + i] = (turn_of ? part[l.c1[u] + i] : 0.f) + dw.b[u][i];
            }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.D; i += kThreads) s.partial[cta * a.D + i] = part[i];
}

// dw of one side (blockIdx.y): the CTAs' rows in order, a warp per element.
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ Args a, float *dw_q, float *dw_k) {
    const Side &s = a.side[blockIdx.y];
    float *dw = blockIdx.y ? dw_k : dw_q;
    const int d = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (!dw || d >= a.D) return;
    float v = 0.f;
    for (int i = threadIdx.x & 31; i < s.ctas; i += 32) v += s.partial[static_cast<int64_t>(i) * a.D + d];
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) dw[d] = v;
}

// ---- host -----------------------------------------------------------------

// Heads of D elements at byte strides {head, token}: as rows of one matrix, and no two
// heads of an output may overlap.
int check_heads(const int64_t nb[2], int64_t D, int64_t H, int64_t T, int size, bool output) {
    const int64_t row = D * size;
    for (int i = 0; i < 2; ++i) {
        const int rc = check_row_stride(row, i ? T : H, nb[i], size, output);
        if (rc != OOP_OK) return rc;
    }
    if (output && H > 1 && T > 1) {
        const bool head_first = nb[0] <= nb[1];
        const int64_t lo = head_first ? nb[0] : nb[1], hi = head_first ? nb[1] : nb[0];
        if (hi < lo * ((head_first ? H : T) - 1) + row) return OOP_ERR_SHAPE;
    }
    return OOP_OK;
}

int check_common(int64_t D, int64_t n_rot, int64_t T, const int32_t *pos, const float *freqs, float eps) {
    if (D < 1 || D > kMaxHead || T < 0 || T > 0x7fffffffLL || n_rot < 0 || n_rot > D || n_rot % 2)
        return OOP_ERR_SHAPE;
    if (!(eps >= 0.f && std::isfinite(eps))) return OOP_ERR_VALUE;
    if (T > 0 && n_rot > 0) {
        int rc = check_pointer(pos, 4);
        if (rc == OOP_OK) rc = check_pointer(freqs, 4);
        if (rc != OOP_OK) return rc;
    }
    return OOP_OK;
}

constexpr int64_t kMaxHeads = 1 << 20;

// Fills in what follows from the sizes; e is the chunk.
void plan(Args &a, int e, int64_t D, int64_t n_rot, int64_t T, int sms, bool backward) {
    a.T = T;
    a.D = static_cast<int>(D);
    a.half = static_cast<int>(n_rot / 2);
    a.inv_d = 1.f / static_cast<float>(D);
    // squares below 2^-126 lose bits: of up to 1024 they matter to a sum below 2^-100
    a.low = static_cast<double>(a.eps) * static_cast<double>(D) < 0x1p-100 ? 0x1p-100f : 0.f;
    a.units = a.half / e + static_cast<int>((D - n_rot + 2 * e - 1) / (2 * e));
    a.group_shift = 0;
    while ((1 << a.group_shift) < a.units && a.group_shift < 5) ++a.group_shift;
    const int64_t groups = 32 >> a.group_shift;
    // a token's heads are split until there are sixteen warps for each SM
    auto splits_of = [&](int64_t heads) {
        const int64_t most = (heads + groups - 1) / groups;
        int64_t n = 1;
        while (n < most && T * n < 16LL * sms) ++n;
        return static_cast<int>(n);
    };
    const int64_t resident = 2LL * sms, warps = kThreads / 32;
    if (!backward) {
        a.side[0].splits = splits_of(std::max(a.side[0].heads, a.side[1].heads));
        a.side[0].ctas = static_cast<int>(std::min<int64_t>(resident, (T * a.side[0].splits + warps - 1) / warps));
        return;
    }
    int64_t items[2] = {0, 0}, cost[2] = {0, 0};
    for (int i = 0; i < 2; ++i) {
        Side &s = a.side[i];
        if (s.heads == 0) continue;                        // no CTAs
        s.splits = splits_of(s.heads);
        items[i] = (T * s.splits + warps - 1) / warps;
        // turns of an item, and about one for its angles
        cost[i] = (s.heads + groups * s.splits - 1) / (groups * s.splits) + 1;
    }
    // the share of the resident CTAs that ends both sides together
    auto rounds = [&](int i, int64_t ctas) { return (items[i] + ctas - 1) / ctas * cost[i]; };
    int64_t best = 0, split = 0;
    for (int64_t n = 1; n < resident; ++n) {
        const int64_t time = std::max(rounds(0, n), rounds(1, resident - n));
        if (!split || time < best) best = time, split = n;
    }
    for (int i = 0; i < 2; ++i)
        if (items[i]) a.side[i].ctas = static_cast<int>(std::min(items[i], !items[1 - i] ? resident : i ? resident - split : split));
}

// The CTAs that have a row of sums: as many as plan() can give one side.
int64_t partial_rows(int64_t T, int64_t H, int sms) {
    return H ? std::max<int64_t>(1, std::min<int64_t>(2LL * sms, T * H)) : 0;
}

template <int TYPE, int E, int U>
void start_forward(const Args &a, cudaStream_t st) {
    forward_kernel<TYPE, E, U><<<a.side[0].ctas, kThreads, 0, st>>>(a);
}
template <int TYPE>
void launch_forward(const Args &a, int e, cudaStream_t st) {
    const int per_lane = (a.units + 31) / 32;
    if constexpr (TYPE != OOP_TYPE_F32) {
        if (e == 8) return per_lane == 1 ? start_forward<TYPE, 8, 1>(a, st) : start_forward<TYPE, 8, 2>(a, st);
    }
    if (e == 4) return per_lane == 1 ? start_forward<TYPE, 4, 1>(a, st) : start_forward<TYPE, 4, 4>(a, st);
    if (per_lane == 1) return start_forward<TYPE, 1, 1>(a, st);
    return per_lane <= 4 ? start_forward<TYPE, 1, 4>(a, st) : start_forward<TYPE, 1, 16>(a, st);
}

template <int DTYPE, int TYPE, int E, int U>
void start_backward(const Args &a, cudaStream_t st) {
    backward_kernel<DTYPE, TYPE, E, U><<<a.side[0].ctas + a.side[1].ctas, kThreads, 0, st>>>(a);
}
template <int DTYPE, int TYPE>
void launch_backward(const Args &a, int e, cudaStream_t st) {
    const int per_lane = (a.units + 31) / 32;
    if constexpr (TYPE != OOP_TYPE_F32 && DTYPE != OOP_TYPE_F32) {
        if (e == 8)
            return per_lane == 1 ? start_backward<DTYPE, TYPE, 8, 1>(a, st) : start_backward<DTYPE, TYPE, 8, 2>(a, st);
    }
    if (e == 4)
        return per_lane == 1 ? start_backward<DTYPE, TYPE, 4, 1>(a, st) : start_backward<DTYPE, TYPE, 4, 4>(a, st);
    if (per_lane == 1) return start_backward<DTYPE, TYPE, 1, 1>(a, st);
    return per_lane <= 4 ? start_backward<DTYPE, TYPE, 1, 4>(a, st) : start_backward<DTYPE, TYPE, 1, 16>(a, st);
}
template <int DTYPE>
void launch_backward_of(const Args &a, int x_type, int e, cudaStream_t st) {
    if (x_type == OOP_TYPE_F32) launch_backward<DTYPE, OOP_TYPE_F32>(a, e, st);
    else if (x_type == OOP_TYPE_F16) launch_backward<DTYPE, OOP_TYPE_F16>(a, e, st);
    else launch_backward<DTYPE, OOP_TYPE_BF16>(a, e, st);
}

// Whether chunks of e elements of this size fit a tensor of heads.
bool chunks_fit(int e, int size, const void *p, int64_t head, int64_t tok, int64_t H, int64_t T) {
    const int bytes = std::min(16, e * size);
    return is_aligned(p, bytes) && (H <= 1 || head % bytes == 0) && (T <= 1 || tok % bytes == 0);
}

}  // namespace
}  // namespace oop

using namespace oop;

extern "C" {

int oop_qk_norm_rope(const oop_heads *q, const oop_heads *k, int type, int w_type, const int32_t *pos,
                     const float *freqs, int64_t D, int64_t n_rot, int64_t T, int interleaved, float eps,
                     void *stream) {
    g_kernel_launches = 0;
    if (!q) return OOP_ERR_NULL;
    const int size = plain_size(type), w_size = plain_size(w_type);
    if (!size || !w_size) return OOP_ERR_TYPE;
    int rc = check_common(D, n_rot, T, pos, freqs, eps);
    if (rc != OOP_OK) return rc;
    Args a = {};
    const oop_heads *in[2] = {q, k};
    for (int i = 0; i < 2; ++i) {
        const oop_heads *p = in[i];
        if (!p) continue;
        if (p->n_head < 0 || p->n_head > kMaxHeads) return OOP_ERR_SHAPE;
        if ((rc = check_heads(p->nb_x, D, p->n_head, T, size, false)) != OOP_OK) return rc;
        if ((rc = check_heads(p->nb_y, D, p->n_head, T, size, true)) != OOP_OK) return rc;
        if (p->n_head == 0 || T == 0) continue;
        if ((rc = check_pointer(p->x, size)) != OOP_OK) return rc;
        if ((rc = check_pointer(p->y, size)) != OOP_OK) return rc;
        if (p->w && !is_aligned(p->w, w_size)) return OOP_ERR_ALIGN;
        Side &s = a.side[i];
        s.x = p->x;
        s.out = p->y;
        s.w = p->w;
        s.x_head = p->nb_x[0], s.x_tok = p->nb_x[1], s.out_head = p->nb_y[0], s.out_tok = p->nb_y[1];
        s.heads = static_cast<int>(p->n_head);
    }
    if (a.side[0].heads + a.side[1].heads == 0) return OOP_OK;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    a.pos = pos;
    a.freqs = freqs;
    a.w_type = w_type;
    a.interleaved = interleaved != 0;
    a.eps = eps;
    auto fits = [&](int e) {
        if ((n_rot / 2) % e || (D - n_rot) % (2 * e)) return false;
        for (const Side &s : a.side)
            if (s.heads && (!chunks_fit(e, size, s.x, s.x_head, s.x_tok, s.heads, T) ||
                            !chunks_fit(e, size, s.out, s.out_head, s.out_tok, s.heads, T)))
                return false;
        return true;
    };
    const int e = size == 2 && fits(8) ? 8 : fits(4) ? 4 : 1;
    plan(a, e, D, n_rot, T, device_sm_count(), false);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (type == OOP_TYPE_F32) launch_forward<OOP_TYPE_F32>(a, e, st);
    else if (type == OOP_TYPE_F16) launch_forward<OOP_TYPE_F16>(a, e, st);
    else launch_forward<OOP_TYPE_BF16>(a, e, st);
    g_kernel_launches = 1;
    return cuda_status(cudaGetLastError());
}

// Room for the rows of sums of both sides on a GPU of up to 160 SMs.
constexpr int kMostSms = 160;

size_t oop_qk_norm_rope_back_workspace_size(int64_t D, int64_t T, int64_t n_head_q, int64_t n_head_k) {
    if (D < 1 || D > kMaxHead || T < 0 || n_head_q < 0 || n_head_k < 0 || n_head_q > kMaxHeads ||
        n_head_k > kMaxHeads || T > 0x7fffffffLL)
        return 0;
    return static_cast<size_t>(partial_rows(T, n_head_q, kMostSms) + partial_rows(T, n_head_k, kMostSms)) *
           static_cast<size_t>(D) * sizeof(float);
}

int oop_qk_norm_rope_back(const oop_heads_grad *q, const oop_heads_grad *k, int dy_type, int x_type,
                          int w_type, const int32_t *pos, const float *freqs, int64_t D, int64_t n_rot,
                          int64_t T, int interleaved, float eps, void *workspace,
                          size_t workspace_bytes, void *stream) {
    g_kernel_launches = 0;
    if (!q) return OOP_ERR_NULL;
    const int size = plain_size(x_type), d_size = plain_size(dy_type), w_size = plain_size(w_type);
    if (!size || !w_size || !gradient_type(dy_type)) return OOP_ERR_TYPE;
    int rc = check_common(D, n_rot, T, pos, freqs, eps);
    if (rc != OOP_OK) return rc;
    Args a = {};
    float *dw[2] = {nullptr, nullptr};
    int64_t heads[2] = {0, 0};
    const oop_heads_grad *in[2] = {q, k};
    for (int i = 0; i < 2; ++i) {
        const oop_heads_grad *p = in[i];
        if (!p) continue;
        if (p->n_head < 0 || p->n_head > kMaxHeads) return OOP_ERR_SHAPE;
        if ((rc = check_heads(p->nb_x, D, p->n_head, T, size, false)) != OOP_OK) return rc;
        if ((rc = check_heads(p->nb_dy, D, p->n_head, T, d_size, false)) != OOP_OK) return rc;
        if ((rc = check_heads(p->nb_dx, D, p->n_head, T, d_size, true)) != OOP_OK) return rc;
        if (p->dw && !is_aligned(p->dw, 4)) return OOP_ERR_ALIGN;
        if (p->w && !is_aligned(p->w, w_size)) return OOP_ERR_ALIGN;
        dw[i] = p->dw;
        heads[i] = p->n_head;
        if (p->n_head == 0 || T == 0) continue;
        if ((rc = check_pointer(p->x, size)) != OOP_OK) return rc;
        if ((rc = check_pointer(p->dy, d_size)) != OOP_OK) return rc;
        if ((rc = check_pointer(p->dx, d_size)) != OOP_OK) return rc;
        Side &s = a.side[i];
        s.x = p->x;
        s.dy = p->dy;
        s.out = p->dx;
        s.w = p->w;
        s.x_head = p->nb_x[0], s.x_tok = p->nb_x[1], s.out_head = p->nb_dx[0], s.out_tok = p->nb_dx[1];
        s.dy_head = p->nb_dy[0], s.dy_tok = p->nb_dy[1];
        s.heads = static_cast<int>(p->n_head);
    }
    const bool any = a.side[0].heads + a.side[1].heads > 0, want = dw[0] || dw[1];
    if (!any && !want) return OOP_OK;
    if (any && want) {
        const size_t need = oop_qk_norm_rope_back_workspace_size(D, T, heads[0], heads[1]);
        if (!workspace || workspace_bytes < need || !is_aligned(workspace, 256)) return OOP_ERR_WORKSPACE;
    }
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!any) {                                            // sums of nothing
        for (float *p : dw)
            if (p && (rc = cuda_status(cudaMemsetAsync(p, 0, static_cast<size_t>(D) * 4, st))) != OOP_OK) return rc;
        return OOP_OK;
    }
    a.pos = pos;
    a.freqs = freqs;
    a.w_type = w_type;
    a.interleaved = interleaved != 0;
    a.eps = eps;
    auto fits = [&](int e) {
        if ((n_rot / 2) % e || (D - n_rot) % (2 * e)) return false;
        for (const Side &s : a.side)
            if (s.heads && (!chunks_fit(e, size, s.x, s.x_head, s.x_tok, s.heads, T) ||
                            !chunks_fit(e, d_size, s.dy, s.dy_head, s.dy_tok, s.heads, T) ||
                            !chunks_fit(e, d_size, s.out, s.out_head, s.out_tok, s.heads, T)))
                return false;
        return true;
    };
    const int e = size == 2 && d_size == 2 && fits(8) ? 8 : fits(4) ? 4 : 1;
    plan(a, e, D, n_rot, T, std::min(device_sm_count(), kMostSms), true);
    float *rows = static_cast<float *>(workspace);
    for (int i = 0; i < 2; ++i) {
        a.side[i].partial = dw[i] ? rows : nullptr;
        if (want) rows += static_cast<int64_t>(a.side[i].ctas) * D;
    }
    if (dy_type == OOP_TYPE_F32) launch_backward_of<OOP_TYPE_F32>(a, x_type, e, st);
    else launch_backward_of<OOP_TYPE_BF16>(a, x_type, e, st);
    if ((rc = cuda_status(cudaGetLastError())) != OOP_OK) return rc;
    g_kernel_launches = 1;
    if (want) {
        const unsigned blocks = static_cast<unsigned>((D + kThreads / 32 - 1) / (kThreads / 32));
        join_kernel<<<dim3(blocks, 2), kThreads, 0, st>>>(a, dw[0], dw[1]);
        g_kernel_launches = 2;
        rc = cuda_status(cudaGetLastError());
    }
    return rc;
}

}  // extern "C"
