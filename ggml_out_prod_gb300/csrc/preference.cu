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
// The paired ratios are sums of small per-token differences, added in 48 bits:
// the difference of two sums of log probabilities would cancel.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "oop_internal.cuh"
#include "rows.cuh"

namespace oop {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;             // 16-byte vectors of one thread and step
constexpr int kJoinThreads = 512;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLog2eRest = 1.92596299112661746887e-8f;    // log2 e - kLog2e
constexpr float kLn2 = 45426.f / 65536.f;                   // log 2 to 16 bits, and the rest
constexpr float kLn2Rest = 1.42860682030941723212e-6f;
// The mean relative error of ex2.approx is -5.0e-8 (measured over [-20, 0], the
// same in every binade), and this is that times -log2 e: added to the
// argument, it keeps long sums of exponentials from coming out low.
constexpr float kNudge = 7.2e-8f;

// Elements of a row that one CTA reads in a step: 16 KB of it.
__host__ __device__ constexpr int64_t step_elems(int size) {
    return int64_t(kThreads) * kVecs * (16 / size);
}
// Steps of a row.  It may start anywhere in a 16-byte vector, so it covers up
// to one vector more than its length.
int64_t steps_of(int64_t V, int size) {
    return std::max<int64_t>(1, (V + 16 / size - 1 + step_elems(size) - 1) / step_elems(size));
}
// CTAs of a row: as few as still give every SM two waves of its four, since a
// CTA keeps the next step's loads in flight through the current one but not
// through its start and end.  (Gradient, bf16, 2300 rows of 32825: 47 us with two
// waves, 52 with four, 61 with eight; forward, f32, 2000 rows of 50257: 57, 56
// and 58.)
constexpr int64_t kWantCtas = 152 * 4 * 2;
int64_t pieces_of(int64_t V, int64_t T, int size) {
    const int64_t steps = steps_of(V, size);
    const int64_t per = std::max<int64_t>(1, steps * T / kWantCtas);
    return (steps + per - 1) / per;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// sum_i exp(x_i) = s * exp(m), m the largest x (or -Inf and s = 0: no terms).
struct LogSum {
    float m, s;
};

// s at a new maximum m >= r.m (equal maxima, infinite ones too, scale by one).
__device__ __forceinline__ float at_max(LogSum r, float m) {
    return r.m == m ? r.s : r.s * expf(r.m - m);
}
__device__ __forceinline__ LogSum join(LogSum a, LogSum b) {
    const float m = fmaxf(a.m, b.m);
    return {m, at_max(a, m) + at_max(b, m)};
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
// One term; a NaN stays in s, where no maximum can lose it, and +Inf is one (Inf - Inf)
// as it is among the vectors.
__device__ __forceinline__ LogSum term(float x) {
    return x < INFINITY ? LogSum{x, 1.f} : LogSum{-INFINITY, x - x};
}
// The join over a warp, scaled once: every factor's error would add up.
__device__ __forceinline__ LogSum warp_join(LogSum r) {
    const float m = warp_max(r.m);
    return {m, warp_sum(at_max(r, m))};
}

// A piece of a row as this thread reads it: vector j of a row is the 16 bytes
// at its j-th 16-byte boundary, counted from the one at or below the row's
// start, so every whole vector is one aligned access whatever the row's
// alignment.  The up to 2 * (E - 1) elements at the row's ends that fill no
// vector are taken one by one by the first threads of the row's first CTA.
template <int XT>
struct Span {
    static constexpr int E = 16 / plain_size(XT);
    static constexpr int kStep = kThreads * kVecs * E;
    const typename Plain<XT>::S *row;
    int first, steps;                // this thread's first element (may be negative)
    unsigned whole;                  // vectors at k < whole (unsigned) lie inside the row
    int edge;                        // this thread's single element, or -1

    __device__ __forceinline__ Span(const void *x, int64_t nb, int64_t t, int piece, int pieces, int V)
        : row(row_of<XT>(x, nb, t)) {
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / plain_size(XT);
        const int all = (V + off + kStep - 1) / kStep, per = (all + pieces - 1) / pieces;
        const int i = static_cast<int>(threadIdx.x);
        steps = max(0, min(all - piece * per, per));
        first = piece * per * kStep + i * E - off;
        whole = static_cast<unsigned>(max(0, V - E + 1));
        const int head = off ? min(E - off, V) : 0, tail = (V - head) % E;
        edge = piece > 0 || i >= head + tail ? -1 : i < head ? i : V - tail + i - head;
    }
    // (no sum here passes 2^31: V is at most 2^30)
    __device__ __forceinline__ int at(int step, int i) const { return first + step * kStep + i * (kThreads * E); }
    __device__ __forceinline__ bool inside(int k) const { return static_cast<unsigned>(k) < whole; }

    // Vectors that are not inside read as -Inf: no probability.
    __device__ __forceinline__ void load(int step, Packed<XT, E> (&raw)[kVecs]) const {
        constexpr uint32_t none = XT == OOP_TYPE_F32   ? 0xff800000u
                                  : XT == OOP_TYPE_F16 ? 0xfc00fc00u
                                                       : 0xff80ff80u;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            raw[i].raw = make_uint4(none, none, none, none);
            if (inside(at(step, i))) raw[i] = load_stream<XT, E>(row + at(step, i));
        }
    }
};

struct Workspace {
    float2 *ratio;       // {2P}: the sum and what its additions lost
    int *done;           // sequences finished
    LogSum *part;        // {pieces, T}
};

Workspace carve(void *ws, int64_t pairs) {
    char *p = static_cast<char *>(ws);
    Workspace w;
    w.done = reinterpret_cast<int *>(p);
    w.ratio = reinterpret_cast<float2 *>(p + 256);
    w.part = reinterpret_cast<LogSum *>(p + 256 + (2 * pairs * 8 + 255) / 256 * 256);
    return w;
}

struct LossArgs {
    const void *x;
    const int32_t *labels, *seq;
    const float *ref;
    float *loss, *losses, *ratios, *logps, *lse;
    int64_t nb_x, V, T, P, pieces;
    double beta, smoothing;
    Workspace ws;
    int *status;
};

// The largest element of a step (NaN aside); 16-bit types two at a time.
template <int XT, int E>
__device__ __forceinline__ float step_max(const Packed<XT, E> (&raw)[kVecs]) {
    if constexpr (XT == OOP_TYPE_F32) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            float v[E];
            raw[i].get(v);
#pragma unroll
            for (int e = 0; e < E; ++e) m = fmaxf(m, v[e]);
        }
        return m;
    } else {
        using Two = std::conditional_t<XT == OOP_TYPE_F16, __half2, __nv_bfloat162>;
        Two w[kVecs * E / 2];
        __builtin_memcpy(w, raw, sizeof w);
#pragma unroll
        for (int n = kVecs * E / 4; n > 0; n /= 2)
#pragma unroll
            for (int i = 0; i < n; ++i) w[i] = __hmax2(w[i], w[i + n]);
        return fmaxf(to_float(w[0].x), to_float(w[0].y));
    }
}

// Adds a step's elements to the thread's sum: their maximum first, then one
// exponential per element against the larger of it and the sum's.  log2 e
// takes two terms: in one, its error times x - m (about -6 where a trained
// model's probability lies) would bias every sum by 1e-7.
template <int XT, int E>
__device__ __forceinline__ void add_step(LogSum &r, const Packed<XT, E> (&raw)[kVecs]) {
    const float m = fmaxf(r.m, step_max<XT, E>(raw));
    const float from = m == -INFINITY ? 0.f : m;
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        float v[E];
        raw[i].get(v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float d = v[e] - from;
            sum[e & 1] += exp2_fast(fmaf(d, kLog2e, fmaf(d, kLog2eRest, kNudge)));
        }
    }
    r = {m, at_max(r, m) + (sum[0] + sum[1])};
}

// Bound by memory: the scored rows are read once.  A CTA reads one piece of a row,
// the loads of the next step in flight while this one's elements are added.
// bf16, 10018 scored rows (8 pairs) of 128000: 373 us, 6.9 TB/s, 101% of the measured
// copy rate, which writes as well (all of a CTA's loads first and 71 registers: 520
// us; a join per element: 1680).
template <int XT>
__global__ void __launch_bounds__(kThreads, 4) loss_part_kernel(const LossArgs a) {
    __shared__ LogSum part[kThreads / 32];
    let_next_start();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ws.done = 0;
    const int pieces = static_cast<int>(a.pieces);
    const int t = blockIdx.x / pieces, c = blockIdx.x - t * pieces;
    const int32_t label = a.labels[t];
    if (label < 0 || label >= a.V) return;
    const Span<XT> span(a.x, a.nb_x, t, c, pieces, static_cast<int>(a.V));
    constexpr int E = Span<XT>::E;
    Packed<XT, E> now[kVecs], next[kVecs];
    LogSum r = {-INFINITY, 0.f};
    if (span.steps > 0) span.load(0, now);
    for (int step = 0; step < span.steps; step += 2) {
        if (step + 1 < span.steps) span.load(step + 1, next);
        add_step(r, now);
        if (step + 1 >= span.steps) break;
        if (step + 2 < span.steps) span.load(step + 2, now);
        add_step(r, next);
    }
    if (span.edge >= 0) r = join(r, term(to_float(span.row[span.edge])));
    r = warp_join(r);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) part[warp] = r;
    __syncthreads();
    if (warp > 0) return;
    r = warp_join(lane < kThreads / 32 ? part[lane] : LogSum{-INFINITY, 0.f});
    if (lane == 0) a.ws.part[static_cast<int64_t>(t) * pieces + c] = r;
}

__device__ __forceinline__ float softplus(float x) {         // log(1 + exp(x))
    return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

// A sum of floats with what its additions lost (Knuth's two-sum): 48 bits at
// fp32 speed, where this GPU's few fp64 units would take microseconds.  The
// two are added at the end only, so an infinite sum stays infinite.
struct TwoSum {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float s = hi + v, t = s - hi;
        lo += (hi - (s - t)) + (v - t);
        hi = s;
    }
    __device__ __forceinline__ void add(TwoSum v) {
        add(v.hi);
        lo += v.lo;
    }
    __device__ __forceinline__ float value() const { return isfinite(hi) ? hi + lo : hi; }
};

// The sum over the CTA, in every thread of warp 0.
__device__ __forceinline__ TwoSum block_sum(TwoSum v, TwoSum *part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto over_lanes = [](TwoSum &r) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            TwoSum other;
            other.hi = __shfl_xor_sync(0xffffffffu, r.hi, o);
            other.lo = __shfl_xor_sync(0xffffffffu, r.lo, o);
            r.add(other);
        }
    };
    over_lanes(v);
    if (lane == 0) part[warp] = v;
    __syncthreads();
    if (warp == 0) {
        v = lane < static_cast<int>(blockDim.x >> 5) ? part[lane] : TwoSum{};
        over_lanes(v);
    }
    return v;
}

// One CTA per sequence joins its rows' partial sums; the last CTA to finish
// takes the pairs.  Without pairs, one CTA per kJoinThreads rows.
template <int XT>
__global__ void __launch_bounds__(kJoinThreads) loss_join_kernel(const LossArgs a) {
    __shared__ TwoSum part[kJoinThreads / 32], part2[kJoinThreads / 32];
    __shared__ bool last;
    const int64_t n_seq = 2 * a.P, s = blockIdx.x;
    int64_t t0 = 0, t1 = 0;            // the rows written here
    int64_t s0 = 0, s1 = 0;            // those of them in the sequence
    if (a.P == 0) {
        t0 = s * kJoinThreads;
        t1 = min(a.T, t0 + kJoinThreads);
    } else {
        const int64_t b0 = a.seq[s], b1 = a.seq[s + 1];
        if (threadIdx.x == 0 && (b0 < 0 || b1 < b0 || b1 > a.T)) record_status(a.status, OOP_ERR_BAD_ID);
        s0 = min(max(b0, int64_t(0)), a.T);
        s1 = min(max(b1, s0), a.T);
        t0 = s == 0 ? 0 : s0;
        t1 = s == n_seq - 1 ? a.T : s1;
    }
    TwoSum sum;
    for (int64_t t = t0 + threadIdx.x; t - threadIdx.x < t1; t += kJoinThreads) {
        int32_t label = -1;
        float ref = 0.f, x = 0.f;
        if (t < t1) {
            label = a.labels[t];
            if (a.ref && label >= 0) ref = a.ref[t];
            if (label >= a.V) record_status(a.status, OOP_ERR_BAD_ID);
            if (label >= 0 && label < a.V) x = to_float(row_of<XT>(a.x, a.nb_x, t)[label]);
        }
        wait_previous();               // the inputs are there; the partial sums may not be yet
        if (t >= t1) break;
        float lse = 0.f, logp = 0.f;
        if (label >= 0 && label < a.V) {
            const LogSum *p = a.ws.part + t * a.pieces;
            LogSum r = p[0];
#pragma unroll 8
            for (int64_t c = 1; c < a.pieces; ++c) r = join(r, p[c]);
            // log(s) = k log 2 + log(f) with s = f 2^k: k times log 2's first 16
            // bits is exact, and log(f) is small, so little is rounded away.
            // All -Inf: no term has been added, and the log is -Inf.
            int k = 0;
            const float f = r.m == -INFINITY && !isnan(r.s) ? 1.f : frexpf(r.s, &k);
            const float z[3] = {k * kLn2, k * kLn2Rest, logf(f)};
            TwoSum lp, all;            // x - m first: m + log(s) may lose log(s)
            lp.add(x);
            lp.add(-r.m);
            all.add(r.m);
            for (int i = 0; i < 3; ++i) {
                lp.add(-z[i]);
                all.add(z[i]);
            }
            lse = all.value();
            logp = lp.value();
            if (t >= s0 && t < s1) {
                lp.add(-ref);
                sum.add(lp);
            }
        }
        a.lse[t] = lse;
        a.logps[t] = logp;
    }
    if (a.P == 0) return;
    wait_previous();                   // (a sequence without rows)
    sum = block_sum(sum, part);
    if (threadIdx.x == 0) {
        const float ratio = sum.value();
        a.ws.ratio[s] = isfinite(ratio) ? make_float2(sum.hi, sum.lo) : make_float2(ratio, 0.f);
        a.ratios[s] = ratio;
        __threadfence();
        last = atomicAdd(a.ws.done, 1) == n_seq - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    TwoSum total;
    for (int64_t i = threadIdx.x; i < a.P; i += kJoinThreads) {
        const float2 chosen = __ldcg(a.ws.ratio + i), other = __ldcg(a.ws.ratio + a.P + i);
        TwoSum d;
        d.add(chosen.x);
        d.add(-other.x);
        d.lo += chosen.y - other.y;
        const float m = static_cast<float>(a.beta * (isfinite(d.hi) ? static_cast<double>(d.hi) + d.lo : d.hi));
        const float e = static_cast<float>(a.smoothing), rest = static_cast<float>(1.0 - a.smoothing);
        // a weight of zero takes no part, whatever it would multiply
        const float l = (rest > 0.f ? rest * softplus(-m) : 0.f) + (e > 0.f ? e * softplus(m) : 0.f);
        a.losses[i] = l;
        total.add(l);
    }
    total = block_sum(total, part2);
    if (threadIdx.x == 0) *a.loss = total.value() / static_cast<float>(a.P);
}

struct LossBackArgs {
    const void *x;
    const int32_t *labels, *seq;
    const float *lse, *ratios, *dloss;
    void *dx;
    int64_t nb_x, nb_dx, V, T, P, pieces;
    double beta, smoothing, scale;                // scale: beta / P
    int *status;
};

// d(loss) / d(logp) of a row of sequence s.  In 64 bits, so that a small
// difference of the two terms keeps its digits, but in as few of this GPU's slow
// 64-bit operations as that takes: one exponential (the Taylor series to the 8th
// power on [-0.35, 0.35], off by 2e-10) and one reciprocal (a 32-bit one and a
// Newton step) give both sigma(m) and sigma(-m).
__device__ __forceinline__ float slope_of(const LossBackArgs &a, int64_t s) {
    const int64_t i = s < a.P ? s : s - a.P;
    const double m = a.beta * (static_cast<double>(a.ratios[i]) - a.ratios[a.P + i]), size = fabs(m);
    double t = size;                              // exp(-|m|); NaN stays NaN
    if (size < 700.0) {
        const int k = __float2int_rn(static_cast<float>(size) * kLog2e);
        const double r = fma(static_cast<double>(k), 0.69314718055994530942, -size);
        t = 1.0 / 40320.0;
        t = fma(t, r, 1.0 / 5040.0);
        t = fma(t, r, 1.0 / 720.0);
        t = fma(t, r, 1.0 / 120.0);
        t = fma(t, r, 1.0 / 24.0);
        t = fma(t, r, 1.0 / 6.0);
        t = fma(t, r, 0.5);
        t = fma(t, r, 1.0);
        t = fma(t, r, 1.0) * __longlong_as_double(static_cast<long long>(1023 - k) << 52);
    } else if (size >= 700.0) {
        t = 0.0;
    }
    const double both = 1.0 + t;
    const double guess = 1.f / static_cast<float>(both);
    const double large = guess * fma(-both, guess, 2.0), small = t * large;    // sigma(|m|), sigma(-|m|)
    const double pos = m < 0.0 ? small : large, neg = m < 0.0 ? large : small;
    const double up = a.dloss ? static_cast<double>(*a.dloss) : 1.0;
    const double c = up * a.scale * (a.smoothing * pos - (1.0 - a.smoothing) * neg);
    return static_cast<float>(s < a.P ? c : -c);
}

// The sequence that holds row t, or -1: the last s with seq[s] <= t.  A warp
// searches 32 places at a time: two steps for up to 1023 sequences.
__device__ __forceinline__ int64_t sequence_of(const LossBackArgs &a, int64_t t) {
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, n = 2 * a.P + 1;              // the answer's successor lies in lo .. lo + n
    while (n > 0) {
        const int64_t step = (n + 31) / 32;
        const int64_t k = lo + step * (lane + 1) - 1;
        const bool below = k < lo + n && a.seq[k] <= t;
        const int first = __popc(__ballot_sync(0xffffffffu, below));   // steps wholly at or below t
        const int64_t end = lo + n;
        lo += step * first;
        n = min(step - 1, end - lo);
        if (lo >= end) n = 0;
    }
    return lo - 1 < 2 * a.P ? lo - 1 : -1;
}

// Bound by memory: scored rows are read once, all rows are written once.  A CTA
// takes one piece of a row, as in the forward pass.  bf16, 6984 rows (4 pairs) of
// 50257, whose rows are not aligned: 188 us, 6.5 TB/s (96% of the measured copy
// rate); with the ends of rows read by a slow path of every thread, 294.
template <int XT, int DT>
__global__ void __launch_bounds__(kThreads, 4) loss_back_kernel(const LossBackArgs a) {
    __shared__ float coef;
    const int pieces = static_cast<int>(a.pieces);
    const int t = blockIdx.x / pieces, c = blockIdx.x - t * pieces;
    const int32_t label = a.labels[t];
    const bool scored = label >= 0 && label < a.V && a.P > 0;
    const Span<XT> span(a.x, a.nb_x, t, c, pieces, static_cast<int>(a.V));
    constexpr int E = Span<XT>::E, kOut = E * plain_size(DT) < 16 ? E * plain_size(DT) : 16;
    Packed<XT, E> now[kVecs], next[kVecs];
    float lse = 0.f;
    if (scored) {
        lse = a.lse[t];
        if (span.steps > 0) span.load(0, now);
    }
    if (threadIdx.x < 32) {                       // while the row is on its way
        const int64_t s = scored ? sequence_of(a, t) : -1;
        if (threadIdx.x == 0) {
            if (label >= a.V) record_status(a.status, OOP_ERR_BAD_ID);
            coef = s >= 0 ? slope_of(a, s) : 0.f;
        }
    }
    __syncthreads();
    const float k = coef;
    auto *dx = row_of<DT>(a.dx, a.nb_dx, t);
    const bool aligned = (reinterpret_cast<uintptr_t>(dx + span.first) & (kOut - 1)) == 0;
    auto put = [&](int at, const float (&v)[E]) {
        if (!span.inside(at)) return;
        if (aligned) {
            store_stream<DT, E>(dx + at, v);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) dx[at + e] = from_float<DT>(v[e]);
        }
    };
    if (!scored || k == 0.f) {
        float zero[E];
#pragma unroll
        for (int e = 0; e < E; ++e) zero[e] = 0.f;
        for (int step = 0; step < span.steps; ++step)
#pragma unroll
            for (int i = 0; i < kVecs; ++i) put(span.at(step, i), zero);
        if (span.edge >= 0) dx[span.edge] = from_float<DT>(0.f);
        return;
    }
    auto slope = [&](float x, int at) {
        const float v = -k * exp2_fast((x - lse) * kLog2e);
        return at == label ? v + k : v;
    };
    if (span.edge >= 0) dx[span.edge] = from_float<DT>(slope(to_float(span.row[span.edge]), span.edge));
    auto do_step = [&](int step, const Packed<XT, E> (&raw)[kVecs]) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int at = span.at(step, i);
            float v[E];
            raw[i].get(v);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = -k * exp2_fast((v[e] - lse) * kLog2e);
            if (label >= at && label < at + E) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (label == at + e) v[e] += k;
            }
            put(at, v);
        }
    };
    for (int step = 0; step < span.steps; step += 2) {
        if (step + 1 < span.steps) span.load(step + 1, next);
        do_step(step, now);
        if (step + 1 >= span.steps) break;
        if (step + 2 < span.steps) span.load(step + 2, now);
        do_step(step + 1, next);
    }
}

int check_loss(const int64_t ne[2], int64_t pairs) {
    if (!ne) return OOP_ERR_NULL;
    const int rc = check_extent(ne[0], ne[1]);
    if (rc != OOP_OK) return rc;
    if (pairs < 0 || pairs > 0x3fffffffLL || ne[0] > (1 << 30) || ne[1] > 0x7fffffffLL)
        return OOP_ERR_SHAPE;
    if (steps_of(ne[0], 4) * ne[1] > 0x7fffffffLL) return OOP_ERR_SHAPE;    // CTAs ride grid.x
    return OOP_OK;
}

int check_scalars(double beta, double smoothing) {
    return std::isfinite(beta) && smoothing >= 0.0 && smoothing <= 1.0 ? OOP_OK : OOP_ERR_VALUE;
}

template <int XT>
cudaError_t launch_loss(const LossArgs &a, cudaStream_t st) {
    if (a.T > 0) loss_part_kernel<XT><<<static_cast<unsigned>(a.T * a.pieces), kThreads, 0, st>>>(a);
    const int64_t grid = a.P > 0 ? 2 * a.P : (a.T + kJoinThreads - 1) / kJoinThreads;
    return launch_dependent(loss_join_kernel<XT>, dim3(static_cast<unsigned>(grid)), kJoinThreads, 0,
                            st, a);
}

}  // namespace
}  // namespace oop

using namespace oop;

extern "C" {

size_t oop_preference_loss_workspace_size(const int64_t ne[2], int64_t n_pairs) {
    if (check_loss(ne, n_pairs) != OOP_OK) return 0;
    return 256 + static_cast<size_t>(2 * n_pairs * 8 + 255) / 256 * 256 +
           static_cast<size_t>(ne[1] * std::max(pieces_of(ne[0], ne[1], 4), pieces_of(ne[0], ne[1], 2))) *
               sizeof(LogSum);
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
                        n_pairs, pieces_of(V, T, size), beta, label_smoothing, carve(workspace, n_pairs),
                        status};
    cudaError_t e = cudaSuccess;
    if (T == 0) e = cudaMemsetAsync(a.ws.done, 0, sizeof(int), st);
    if (e != cudaSuccess) return cuda_status(e);
    e = type == OOP_TYPE_F32   ? launch_loss<OOP_TYPE_F32>(a, st)
        : type == OOP_TYPE_F16 ? launch_loss<OOP_TYPE_F16>(a, st)
                               : launch_loss<OOP_TYPE_BF16>(a, st);
    if (e == cudaSuccess) e = cudaGetLastError();
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
                            n_pairs, pieces_of(V, T, size), beta, label_smoothing,
                            n_pairs > 0 ? beta / static_cast<double>(n_pairs) : 0.0, status};
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
    kern<<<static_cast<unsigned>(T * a.pieces), kThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) g_kernel_launches = 1;
    return cuda_status(e);
}

}  // extern "C"
