// rows.cuh -- what the row-wise training operators share: the plain element
// types, vectors of them, reductions over a warp, and the host checks of a
// {M, T} matrix given by a pointer and the byte stride between its rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>

#include "oop_internal.cuh"

namespace oop {

// Bytes of an element of a plain type; 0 for any other type.
__host__ __device__ constexpr int plain_size(int type) {
    return type == OOP_TYPE_F32 ? 4 : (type == OOP_TYPE_F16 || type == OOP_TYPE_BF16) ? 2 : 0;
}

// The types a gradient may have: binary16 overflows at 65504, which
// training gradients pass ("metal: OUT_PROD multiplies in float staging",
// opening paragraph), so it is not one of them.
inline bool gradient_type(int type) { return type == OOP_TYPE_F32 || type == OOP_TYPE_BF16; }

// ---- host checks ----------------------------------------------------------

inline bool is_aligned(const void *p, uintptr_t n) {
    return reinterpret_cast<uintptr_t>(p) % n == 0;
}

// Sizes of a matrix of T rows of `row_bytes` bytes, `nb` bytes apart, of
// elements of `size` bytes: strides are non-negative multiples of the element
// size; the rows of an output must not overlap (0 repeats an input's row).
inline int check_row_stride(int64_t row_bytes, int64_t T, int64_t nb, int size, bool output) {
    if (nb < 0 || nb % size != 0) return OOP_ERR_SHAPE;
    if (output && T > 1 && nb < row_bytes) return OOP_ERR_SHAPE;
    if (static_cast<double>(T) * static_cast<double>(nb > row_bytes ? nb : row_bytes) > 9.0e18)
        return OOP_ERR_SHAPE;
    return OOP_OK;
}

// {M, T} of a call: non-negative, and small enough for int64 byte offsets.
inline int check_extent(int64_t M, int64_t T) {
    if (M < 0 || T < 0) return OOP_ERR_SHAPE;
    if (static_cast<double>(M) * static_cast<double>(T) * 8.0 > 9.0e18) return OOP_ERR_SHAPE;
    return OOP_OK;
}

inline int check_pointer(const void *p, int size) {
    if (!p) return OOP_ERR_NULL;
    return is_aligned(p, static_cast<uintptr_t>(size)) ? OOP_OK : OOP_ERR_ALIGN;
}

// ---- elements -------------------------------------------------------------

template <int TYPE> struct Plain;
template <> struct Plain<OOP_TYPE_F32> { using S = float; };
template <> struct Plain<OOP_TYPE_F16> { using S = __half; };
template <> struct Plain<OOP_TYPE_BF16> { using S = __nv_bfloat16; };

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// Rounded to nearest even; binary16 rounds what lies beyond its range to Inf.
template <int TYPE>
__device__ __forceinline__ typename Plain<TYPE>::S from_float(float v) {
    if constexpr (TYPE == OOP_TYPE_F32) return v;
    else if constexpr (TYPE == OOP_TYPE_F16) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// Element m of a row of a type known at run time (the same for every thread).
__device__ __forceinline__ float load_any(const void *p, int type, int64_t m) {
    if (type == OOP_TYPE_F32) return static_cast<const float *>(p)[m];
    if (type == OOP_TYPE_F16) return __half2float(static_cast<const __half *>(p)[m]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[m]);
}

template <int TYPE>
__device__ __forceinline__ const typename Plain<TYPE>::S *row_of(const void *p, int64_t nb,
                                                                 int64_t t) {
    return reinterpret_cast<const typename Plain<TYPE>::S *>(static_cast<const char *>(p) + t * nb);
}
template <int TYPE>
__device__ __forceinline__ typename Plain<TYPE>::S *row_of(void *p, int64_t nb, int64_t t) {
    return reinterpret_cast<typename Plain<TYPE>::S *>(static_cast<char *>(p) + t * nb);
}

// ---- vectors --------------------------------------------------------------

// E consecutive elements as they lie in memory: 2 to 16 bytes in one access
// (E = 1: the element itself).
template <int BYTES> struct Words;
template <> struct Words<2> { using T = uint16_t; };
template <> struct Words<4> { using T = uint32_t; };
template <> struct Words<8> { using T = uint2; };
template <> struct Words<16> { using T = uint4; };

template <int TYPE, int E>
struct Packed {
    static constexpr int kBytes = E * plain_size(TYPE);
    typename Words<kBytes>::T raw;

    __device__ __forceinline__ void get(float (&v)[E]) const {
        using S = typename Plain<TYPE>::S;
        if constexpr (TYPE == OOP_TYPE_BF16 && E >= 2) {
            uint32_t w[kBytes / 4];
            __builtin_memcpy(w, &raw, kBytes);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {      // a bfloat16 is the top half of its float
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            S e[E];
            __builtin_memcpy(e, &raw, kBytes);
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = to_float(e[i]);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[E]) {
        if constexpr (TYPE == OOP_TYPE_BF16 && E >= 2) {
            __nv_bfloat162 e[E / 2];
#pragma unroll
            for (int i = 0; i < E / 2; ++i) e[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            __builtin_memcpy(&raw, e, kBytes);
        } else if constexpr (TYPE == OOP_TYPE_F16 && E >= 2) {
            __half2 e[E / 2];
#pragma unroll
            for (int i = 0; i < E / 2; ++i) e[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            __builtin_memcpy(&raw, e, kBytes);
        } else {
            typename Plain<TYPE>::S e[E];
#pragma unroll
            for (int i = 0; i < E; ++i) e[i] = from_float<TYPE>(v[i]);
            __builtin_memcpy(&raw, e, kBytes);
        }
    }
};

// Streaming accesses (data read or written once): evicted first, and
// 16-byte loads leave L1 to what is read again (parameters).  Volatile: an
// output may lie over the input, so no load may be repeated later.
template <int TYPE, int E>
__device__ __forceinline__ Packed<TYPE, E> load_stream(const typename Plain<TYPE>::S *p) {
    Packed<TYPE, E> r;
    if constexpr (E * plain_size(TYPE) == 16)
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.raw.x), "=r"(r.raw.y), "=r"(r.raw.z), "=r"(r.raw.w)
                     : "l"(p));
    else
        r.raw = __ldcs(reinterpret_cast<const typename Words<E * plain_size(TYPE)>::T *>(p));
    return r;
}
template <int TYPE, int E>
__device__ __forceinline__ Packed<TYPE, E> load_packed(const typename Plain<TYPE>::S *p) {
    Packed<TYPE, E> r;
    r.raw = *reinterpret_cast<const typename Words<E * plain_size(TYPE)>::T *>(p);
    return r;
}
// E floats as TYPE; more than 16 bytes go in 16-byte pieces.
template <int TYPE, int E>
__device__ __forceinline__ void store_stream(typename Plain<TYPE>::S *p, const float (&v)[E]) {
    if constexpr (E * plain_size(TYPE) > 16) {
        constexpr int H = 16 / plain_size(TYPE);
#pragma unroll
        for (int i = 0; i < E; i += H) {
            float part[H];
#pragma unroll
            for (int j = 0; j < H; ++j) part[j] = v[i + j];
            store_stream<TYPE, H>(p + i, part);
        }
    } else {
        Packed<TYPE, E> r;
        r.set(v);
        __stcs(reinterpret_cast<typename Words<E * plain_size(TYPE)>::T *>(p), r.raw);
    }
}

// ---- launches -------------------------------------------------------------

// Lets KERNEL be launched with all the dynamic shared memory a CTA can have.  The
// call costs about a microsecond, so it is made once per device (two threads
// that race make it twice, with the same value).
constexpr int kMostSmem = 227 * 1024;

template <auto KERNEL>
cudaError_t allow_smem() {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kDevices;
    if (known && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    cudaFuncAttributes attr = {};
    e = cudaFuncGetAttributes(&attr, KERNEL);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kMostSmem - static_cast<int>(attr.sharedSizeBytes));
    if (e == cudaSuccess && known) done[dev].store(true, std::memory_order_relaxed);
    return e;
}

// ---- dependent launches ---------------------------------------------------
//
// A kernel launched with launch_dependent may start while the one before it on
// the stream still runs: as soon as every CTA of that one has called
// let_next_start (or ended).  wait_previous returns once the previous grid has
// ended and its writes are visible; nothing that grid writes may be touched
// before.  A kernel launched plainly waits for everything before it.

__device__ __forceinline__ void let_next_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                             cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- reductions (every lane gets the result; fixed order) -----------------

template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The sum over a CTA of up to 32 warps; `part` holds 32 values.  Every thread
// of the CTA calls it.
template <class T>
__device__ __forceinline__ T block_sum(T v, T *part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int warps = (blockDim.x + 31) >> 5;
    v = warp_sum(v);
    __syncthreads();          // part may still be read by an earlier call
    if (lane == 0) part[warp] = v;
    __syncthreads();
    return warp_sum(lane < warps ? part[lane] : T(0));
}

}  // namespace oop
