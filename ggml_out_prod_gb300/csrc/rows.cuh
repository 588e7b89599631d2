// rows.cuh -- what the row-wise training operators share: the plain element
// types, vectors of them, reductions over a warp, and the host checks of a
// {M, T} matrix given by a pointer and the byte stride between its rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
