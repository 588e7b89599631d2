// gated_ffn.cu -- the gated feed-forward block up to its last projection, and
// its backward pass.
//
//   gate = x Wg',  up = x Wu',  h = act(gate) up
//   dgate = dh up act'(gate),  dup = dh act(gate)
//   dx = dgate Wg + dup Wu,  dWg = dgate' x,  dWu = dup' x
#include <algorithm>
#include <cmath>

#include "oop_internal.cuh"
#include "products.cuh"
#include "rows.cuh"

namespace oop {
namespace {

constexpr float kGelu = 0.7978845608028654f;               // sqrt(2 / pi)

// The activation and its derivative.
template <bool SLOPE>
__device__ __forceinline__ float activation(float v, int act, float &slope) {
    if (act == OOP_ACT_SILU) {
        const float s = 1.f / (1.f + expf(-v));
        if (SLOPE) slope = s * (1.f + v * (1.f - s));
        return v * s;
    }
    if (act == OOP_ACT_GELU_TANH) {
        const float t = tanhf(kGelu * (v + 0.044715f * v * v * v));
        if (SLOPE) slope = 0.5f * (1.f + t) + 0.5f * v * (1.f - t * t) * kGelu * (1.f + 0.134145f * v * v);
        return 0.5f * v * (1.f + t);
    }
    if (act == OOP_ACT_GELU_ERF) {
        const float e = 0.5f * erfcf(-v * 0.7071067811865476f);
        if (SLOPE) slope = e + v * expf(-0.5f * v * v) * 0.3989422804014327f;
        return v * e;
    }
    if (SLOPE) slope = v > 0.f ? 1.f : v == v ? 0.f : v;
    return v > 0.f ? v : v == v ? 0.f : v;
}

struct Rows {
    const void *p;
    int64_t nb;
};

// h and the kept projections from the sums (gate in g, up in u, dense).
template <int TYPE>
__global__ void gate_kernel(const float *g, const float *u, char *h, int64_t nb_h, char *gate, char *up, int64_t nb_gu,
                            int64_t F, int64_t T, int act) {
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < F * T; i += gridDim.x * 256LL) {
        const int64_t t = i / F, f = i - t * F;
        float none;
        row_of<TYPE>(h, nb_h, t)[f] = from_float<TYPE>(activation<false>(g[i], act, none) * u[i]);
        if (gate) {
            row_of<TYPE>(gate, nb_gu, t)[f] = from_float<TYPE>(g[i]);
            row_of<TYPE>(up, nb_gu, t)[f] = from_float<TYPE>(u[i]);
        }
    }
}

__global__ void gate_back_kernel(Rows dh, int d_type, Rows gate, Rows up, int x_type, float *dg, float *du, int64_t F,
                                 int64_t T, int act) {
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < F * T; i += gridDim.x * 256LL) {
        const int64_t t = i / F, f = i - t * F;
        const float d = load_any(static_cast<const char *>(dh.p) + t * dh.nb, d_type, f);
        const float g = load_any(static_cast<const char *>(gate.p) + t * gate.nb, x_type, f);
        const float u = load_any(static_cast<const char *>(up.p) + t * up.nb, x_type, f);
        float slope;
        const float a = activation<true>(g, act, slope);
        float vg = d * u * slope, vu = d * a;
        if (d_type == OOP_TYPE_BF16) {
            vg = __bfloat162float(__float2bfloat16_rn(vg));
            vu = __bfloat162float(__float2bfloat16_rn(vu));
        }
        dg[i] = vg;
        du[i] = vu;
    }
}

template <int TYPE>
__global__ void store_kernel(const float *src, char *dst, int64_t nb, int64_t cols, int64_t rows) {
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < cols * rows; i += gridDim.x * 256LL) {
        const int64_t r = i / cols;
        row_of<TYPE>(dst, nb, r)[i - r * cols] = from_float<TYPE>(src[i]);
    }
}

unsigned blocks_of(int64_t n) { return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((n + 255) / 256, 1 << 18))); }

void store(const float *src, void *dst, int type, int64_t nb, int64_t cols, int64_t rows, cudaStream_t st) {
    char *d = static_cast<char *>(dst);
    if (type == OOP_TYPE_F32) store_kernel<OOP_TYPE_F32><<<blocks_of(cols * rows), 256, 0, st>>>(src, d, nb, cols, rows);
    else store_kernel<OOP_TYPE_BF16><<<blocks_of(cols * rows), 256, 0, st>>>(src, d, nb, cols, rows);
    ++g_kernel_launches;
}

// Floats of the workspace: x, both weights, and two matrices {F, T}; back: and the larger result.
size_t floats_forward(const int64_t ne[3]) {
    return static_cast<size_t>(ne[0] * ne[2] + 2 * ne[0] * ne[1] + 2 * ne[1] * ne[2]);
}
size_t floats_back(const int64_t ne[3]) {
    return floats_forward(ne) + static_cast<size_t>(std::max(ne[0] * ne[2], ne[0] * ne[1]));
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

int check_workspace(const void *ws, size_t have, size_t need) {
    return need == 0 || (ws && have >= need && is_aligned(ws, 256)) ? OOP_OK : OOP_ERR_WORKSPACE;
}

}  // namespace
}  // namespace oop

using namespace oop;

extern "C" {

size_t oop_gated_ffn_workspace_size(int x_type, int w_type, const int64_t ne[3], int aligned) {
    (void)aligned;
    if (check_ffn(x_type, w_type, ne, 0) != OOP_OK) return 0;
    return floats_forward(ne) * 4;
}

size_t oop_gated_ffn_back_workspace_size(int dh_type, int x_type, int w_type, const int64_t ne[3], int aligned) {
    (void)aligned;
    if (!gradient_type(dh_type) || check_ffn(x_type, w_type, ne, 0) != OOP_OK) return 0;
    return floats_back(ne) * 4;
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
    if ((rc = check_workspace(workspace, workspace_bytes, oop_gated_ffn_workspace_size(x_type, w_type, ne, 0))) != OOP_OK)
        return rc;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *xf = static_cast<float *>(workspace), *wf[2] = {xf + K * T, xf + K * T + K * F}, *s[2];
    s[0] = wf[1] + K * F;
    s[1] = s[0] + F * T;
    const void *w[2] = {w_gate, w_up};
    cudaError_t e = launch_to_f32(x, x_type, nb_x, K, T, xf, K, st);
    for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
        e = launch_to_f32(w[i], w_type, nb_w, K, F, wf[i], K, st);
        if (e == cudaSuccess) e = launch_product({xf, wf[i], s[i], T, F, K, 1, K, 1, 0, K, 1, 0, F, 0, 1.f, 0.f}, st);
    }
    if (e != cudaSuccess) return cuda_status(e);
    char *hp = static_cast<char *>(h), *gp = static_cast<char *>(gate), *up_ = static_cast<char *>(up);
    if (x_type == OOP_TYPE_F32) gate_kernel<OOP_TYPE_F32><<<blocks_of(F * T), 256, 0, st>>>(s[0], s[1], hp, nb_h, gp, up_, nb_gu, F, T, act);
    else if (x_type == OOP_TYPE_F16) gate_kernel<OOP_TYPE_F16><<<blocks_of(F * T), 256, 0, st>>>(s[0], s[1], hp, nb_h, gp, up_, nb_gu, F, T, act);
    else gate_kernel<OOP_TYPE_BF16><<<blocks_of(F * T), 256, 0, st>>>(s[0], s[1], hp, nb_h, gp, up_, nb_gu, F, T, act);
    ++g_kernel_launches;
    return cuda_status(cudaGetLastError());
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
    if ((rc = check_workspace(workspace, workspace_bytes, oop_gated_ffn_back_workspace_size(dh_type, x_type, w_type, ne, 0))) != OOP_OK)
        return rc;
    int *status = nullptr;
    if ((rc = device_status_word(&status)) != OOP_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *xf = static_cast<float *>(workspace), *wf[2] = {xf + K * T, xf + K * T + K * F}, *d[2], *out;
    d[0] = wf[1] + K * F;
    d[1] = d[0] + F * T;
    out = d[1] + F * T;
    if (F * T > 0) {
        gate_back_kernel<<<blocks_of(F * T), 256, 0, st>>>({dh, nb_dh}, dh_type, {gate, nb_gu}, {up, nb_gu}, x_type, d[0],
                                                           d[1], F, T, act);
        ++g_kernel_launches;
    }
    cudaError_t e = cudaGetLastError();
    const void *w[2] = {w_gate, w_up};
    if (want_dx) {
        for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
            e = launch_to_f32(w[i], w_type, nb_w, K, F, wf[i], K, st);
            if (e == cudaSuccess)
                e = launch_product({d[i], wf[i], out, T, K, F, 1, F, 1, 0, 1, K, 0, K, 0, 1.f, i ? 1.f : 0.f}, st);
        }
        if (e != cudaSuccess) return cuda_status(e);
        store(out, dx, dh_type, nb_dx, K, T, st);
    }
    if (want_dw) {
        e = launch_to_f32(x, x_type, nb_x, K, T, xf, K, st);
        void *dw[2] = {dw_gate, dw_up};
        for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
            e = launch_product({d[i], xf, out, F, K, T, 1, 1, F, 0, 1, K, 0, K, 0, 1.f, 0.f}, st);
            if (e == cudaSuccess) store(out, dw[i], dh_type, nb_dw, K, F, st);
        }
    }
    return cuda_status(e == cudaSuccess ? cudaGetLastError() : e);
}

}  // extern "C"
