// get_rows.cu -- embedding lookup from a plain or block-quantised table, and
// the gradient of the table.
//
//   y[m, t]  = scale * W[m, ids[t]]
//   dW[m, v] = scale * sum over the t with ids[t] == v of dy[m, t]
//
// (ggml's GET_ROWS and GET_ROWS_BACK; the latter is among the training
// operations that "metal: OUT_PROD runs batched, broadcast and narrow shapes
// on the GPU" lists as still running on the CPU.)
#include "oop_internal.cuh"
#include "quant.cuh"
#include "rows.cuh"

namespace oop {
namespace {

constexpr int kThreads = 256;

template <int TYPE, int OUT>
__global__ void __launch_bounds__(kThreads) get_rows_kernel(const void *table, int64_t nb_table,
                                                            const int32_t *ids, void *dst,
                                                            int64_t nb_dst, int64_t M, int64_t V,
                                                            float scale, int *status) {
    const int64_t t = blockIdx.x;
    const int32_t id = ids[t];
    auto *out = row_of<OUT>(dst, nb_dst, t);
    if (id < 0 || id >= V) {
        for (int64_t m = threadIdx.x; m < M; m += kThreads) out[m] = from_float<OUT>(0.f);
        if (threadIdx.x == 0) record_status(status, OOP_ERR_BAD_ID);
        return;
    }
    const uint8_t *row = static_cast<const uint8_t *>(table) + id * nb_table;
    for (int64_t m = threadIdx.x; m < M; m += kThreads)
        out[m] = from_float<OUT>(scale * decode_row<TYPE>(row, m));
}

// One CTA per table row: the ids are scanned in ascending t, so every sum has
// one order, taken in runs of 64 terms.
template <int TYPE>
__global__ void __launch_bounds__(kThreads) get_rows_back_kernel(const void *dy, int64_t nb_dy,
                                                                 const int32_t *ids, float *dw,
                                                                 int64_t M, int64_t V, int64_t T,
                                                                 float scale, int accumulate,
                                                                 int *status) {
    const int64_t v = blockIdx.x;
    if (v == 0)
        for (int64_t t = threadIdx.x; t < T; t += kThreads)
            if (ids[t] < 0 || ids[t] >= V) record_status(status, OOP_ERR_BAD_ID);
    for (int64_t m = threadIdx.x; m < M; m += kThreads) {
        float sum = 0.f, run = 0.f;
        int n = 0;
        for (int64_t t = 0; t < T; ++t) {
            if (ids[t] != v) continue;
            run += to_float(row_of<TYPE>(dy, nb_dy, t)[m]);
            if (++n % 64 == 0) {
                sum += run;
                run = 0.f;
            }
        }
        sum += run;
        float *out = dw + v * M + m;
        *out = accumulate ? *out + scale * sum : scale * sum;
    }
}

using RowsKernel = void (*)(const void *, int64_t, const int32_t *, void *, int64_t, int64_t,
                            int64_t, float, int *);

template <int TYPE>
RowsKernel rows_kernel(int out) {
    switch (out) {
    case OOP_TYPE_F32: return get_rows_kernel<TYPE, OOP_TYPE_F32>;
    case OOP_TYPE_F16: return get_rows_kernel<TYPE, OOP_TYPE_F16>;
    case OOP_TYPE_BF16: return get_rows_kernel<TYPE, OOP_TYPE_BF16>;
    default: return nullptr;
    }
}

RowsKernel rows_kernel(int type, int out) {
    switch (type) {
#define OOP_ROWS_CASE(T) \
    case T: return rows_kernel<T>(out);
    OOP_ROWS_CASE(OOP_TYPE_F32)
    OOP_ROWS_CASE(OOP_TYPE_F16)
    OOP_ROWS_CASE(OOP_TYPE_BF16)
    OOP_ROWS_CASE(OOP_TYPE_Q4_0)
    OOP_ROWS_CASE(OOP_TYPE_Q4_1)
    OOP_ROWS_CASE(OOP_TYPE_Q5_0)
    OOP_ROWS_CASE(OOP_TYPE_Q5_1)
    OOP_ROWS_CASE(OOP_TYPE_Q8_0)
    OOP_ROWS_CASE(OOP_TYPE_Q2_K)
    OOP_ROWS_CASE(OOP_TYPE_Q3_K)
    OOP_ROWS_CASE(OOP_TYPE_Q4_K)
    OOP_ROWS_CASE(OOP_TYPE_Q5_K)
    OOP_ROWS_CASE(OOP_TYPE_Q6_K)
#undef OOP_ROWS_CASE
    default: return nullptr;
    }
}

int check_rows(const int64_t ne[2], int64_t n_ids) {
    if (!ne) return OOP_ERR_NULL;
    const int rc = check_extent(ne[0], ne[1]);
    if (rc != OOP_OK) return rc;
    if (n_ids < 0 || n_ids > 0x7fffffffLL || ne[1] > 0x7fffffffLL) return OOP_ERR_SHAPE;
    return check_extent(ne[0], n_ids);
}

}  // namespace
}  // namespace oop

using namespace oop;

extern "C" {

int oop_get_rows(const void *table, int table_type, int64_t nb_table, const int32_t *ids,
                 void *dst, int dst_type, int64_t nb_dst, const int64_t ne_table[2],
                 int64_t n_ids, float scale, void *stream) {
    g_kernel_launches = 0;
    int rc = check_rows(ne_table, n_ids);
    if (rc != OOP_OK) return rc;
    const int qk = type_block_elems(table_type);
    if (qk < 0 || !plain_size(dst_type)) return OOP_ERR_TYPE;
    const int64_t M = ne_table[0], V = ne_table[1];
    if (M % qk != 0) return OOP_ERR_SHAPE;
    const int size = table_type == OOP_TYPE_F32 ? 4 : 2;      // every block is of an even size
    rc = check_row_stride(M / qk * type_block_bytes(table_type), V, nb_table, size, false);
    if (rc != OOP_OK) return rc;
    rc = check_row_stride(M * plain_size(dst_type), n_ids, nb_dst, plain_size(dst_type), true);
    if (rc != OOP_OK) return rc;
    if (M == 0 || n_ids == 0) return OOP_OK;
    if ((rc = check_pointer(dst, plain_size(dst_type))) != OOP_OK) return rc;
    if ((rc = check_pointer(ids, 4)) != OOP_OK) return rc;
    if (V > 0 && (rc = check_pointer(table, size)) != OOP_OK) return rc;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    rows_kernel(table_type, dst_type)<<<static_cast<unsigned>(n_ids), kThreads, 0,
                                        static_cast<cudaStream_t>(stream)>>>(
        table, nb_table, ids, dst, nb_dst, M, V, scale, status);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) g_kernel_launches = 1;
    return cuda_status(e);
}

size_t oop_get_rows_back_workspace_size(const int64_t ne_table[2], int64_t n_ids) {
    if (check_rows(ne_table, n_ids) != OOP_OK) return 0;
    return 0;
}

int oop_get_rows_back(const void *dy, int dy_type, int64_t nb_dy, const int32_t *ids,
                      float *dtable, const int64_t ne_table[2], int64_t n_ids, float scale,
                      int accumulate, void *workspace, size_t workspace_bytes, void *stream) {
    g_kernel_launches = 0;
    int rc = check_rows(ne_table, n_ids);
    if (rc != OOP_OK) return rc;
    if (!gradient_type(dy_type)) return OOP_ERR_TYPE;
    const int64_t M = ne_table[0], V = ne_table[1];
    const int size = plain_size(dy_type);
    rc = check_row_stride(M * size, n_ids, nb_dy, size, false);
    if (rc != OOP_OK) return rc;
    if (M == 0 || V == 0) return OOP_OK;
    if ((rc = check_pointer(dtable, 4)) != OOP_OK) return rc;
    if (n_ids > 0) {
        if ((rc = check_pointer(dy, size)) != OOP_OK) return rc;
        if ((rc = check_pointer(ids, 4)) != OOP_OK) return rc;
    }
    const size_t need = oop_get_rows_back_workspace_size(ne_table, n_ids);
    if (need > 0 && (!workspace || workspace_bytes < need || !is_aligned(workspace, 256)))
        return OOP_ERR_WORKSPACE;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const auto kern = dy_type == OOP_TYPE_F32 ? get_rows_back_kernel<OOP_TYPE_F32>
                                              : get_rows_back_kernel<OOP_TYPE_BF16>;
    kern<<<static_cast<unsigned>(V), kThreads, 0, st>>>(dy, nb_dy, ids, dtable, M, V, n_ids, scale,
                                                        accumulate, status);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) g_kernel_launches = 1;
    return cuda_status(e);
}

}  // extern "C"
