// extern "C" boundary of libgdn2: argument checking, path selection, launches.
// Declarations and the meaning of every argument: include/gdn2.h.
#include <stdint.h>

#include <initializer_list>

#include "gdn2.h"
#include "gdn2_internal.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dim_ok(int d) { return d == 64 || d == 128; }

thread_local long long t_wait_limit = -1;   // gdn2_set_wait_limit

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// width of the residual norm: whole 16-byte vectors in either token type, a row within one block's registers
bool width_ok(int width) { return width > 0 && width % 8 == 0 && width <= 8192; }

int check_ptrs(std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs) {
        if (!p) return GDN2_ERR_NULL;
        if (!aligned16(p)) return GDN2_ERR_ALIGN;
    }
    return GDN2_OK;
}

int check_workspace(const void *workspace, size_t bytes, size_t need) {
    if (!workspace) return GDN2_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GDN2_ERR_ALIGN;
    return bytes < need ? GDN2_ERR_WORKSPACE : GDN2_OK;
}

// arguments that the norms share; the comparison also refuses a NaN
int check_norm(long long rows, float eps, int dtype) {
    if (rows < 0) return GDN2_ERR_SHAPE;
    if (dtype != GDN2_F32 && dtype != GDN2_BF16) return GDN2_ERR_DTYPE;
    return eps >= 0.f && eps <= 1.f ? GDN2_OK : GDN2_ERR_VALUE;
}

// Whether slots of two caches share memory without being one cache: where their ranges meet, they must lie one
// stride apart and between one another.
bool caches_clash(const float *a, long long stride_a, int slots_a, const float *b, long long stride_b, int slots_b,
                  long long floats) {
    if (!slots_a || !slots_b || !floats || a == b) return false;
    const long long apart = ((long long)reinterpret_cast<uintptr_t>(b) - (long long)reinterpret_cast<uintptr_t>(a)) / 4;
    if (apart >= (slots_a - 1) * stride_a + floats || -apart >= (slots_b - 1) * stride_b + floats) return false;
    if (slots_a == 1 && slots_b == 1) return true;
    const long long stride = slots_a == 1 ? stride_b : stride_a;   // one slot has no stride
    if (slots_a > 1 && slots_b > 1 && stride_a != stride_b) return true;
    const long long into = (apart % stride + stride) % stride;
    return into < floats || stride - into < floats;
}

// a cache of states: `num_slots` slots of [H, d_k, d_v] floats, `slot_stride` floats apart
int check_pool(const void *S, long long slot_stride, int num_slots, int H, int K, int V) {
    if (slot_stride < (long long)H * K * V) return GDN2_ERR_SHAPE;
    if (num_slots > 0 && !S) return GDN2_ERR_NULL;
    return aligned16(S) && slot_stride % 4 == 0 ? GDN2_OK : GDN2_ERR_ALIGN;
}

int check_common(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
                 const void *o, int B, int H, int K, int V, int dtype) {
    if (B < 0 || H < 0 || K <= 0 || V <= 0) return GDN2_ERR_SHAPE;
    if (dtype != GDN2_F32 && dtype != GDN2_BF16) return GDN2_ERR_DTYPE;
    if (!dim_ok(K) || !dim_ok(V)) return GDN2_ERR_UNSUPPORTED;
    if (!q || !k || !v || !alpha || !b || !w || !o) return GDN2_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(alpha) || !aligned16(b) || !aligned16(w) ||
        !aligned16(o))
        return GDN2_ERR_ALIGN;
    return GDN2_OK;
}

bool use_tc(int B, int H, int T, int K, int V, int C, int dtype) {
    return gdn2::tc_supported(B, H, T, K, V, C, dtype == GDN2_BF16 ? 1 : 0);
}

// Implementation for these sizes: 0 = CUDA-core two-kernel path; 1 = fused tcgen05 kernel (one CTA
// per chain), for up to 64 chains of fewer than 32 chunks; 2 = two-stage tcgen05 path (intra-chunk
// work parallel over every chunk-head, then the state chain, cut into segments in time when there
// are few long chains), for everything else.
int select_path(int B, int H, int T, int K, int V, int C, int dtype) {
    if (!use_tc(B, H, T, K, V, C, dtype)) return 0;
    const long long chains = (long long)B * H, NC = (T + 63) / 64;
    return chains > 64 || NC >= 32 ? 2 : 1;
}

}  // namespace

namespace gdn2 {
uint32_t wait_limit(uint32_t usual) { return t_wait_limit < 0 ? usual : (uint32_t)t_wait_limit; }
}  // namespace gdn2

extern "C" {

size_t gdn2_chunk_fwd_workspace_bytes(int B, int H, int T, int d_k, int d_v, int C, int dtype) {
    if (B < 0 || H < 0 || T < 0 || !dim_ok(d_k) || !dim_ok(d_v) || C != 64) return gdn2::kStatusBytes;
    switch (select_path(B, H, T, d_k, d_v, C, dtype)) {
        case 2: return gdn2::split_workspace_bytes(B, H, T);
        case 1: return gdn2::tc_workspace_bytes(B, H, T, d_k, d_v, C);
        default: return gdn2::simt_workspace_bytes(B, H, T, d_k, d_v, C);
    }
}

size_t gdn2_chunk_fwd_edges_workspace_bytes(int B, int H, int T, int d_k, int d_v, int C) {
    if (B < 0 || H < 0 || T < 0 || !use_tc(B, H, T, d_k, d_v, C, GDN2_BF16)) return gdn2::kStatusBytes;
    if (select_path(B, H, T, d_k, d_v, C, GDN2_BF16) == 2) return gdn2::split_workspace_bytes(B, H, T);
    return gdn2::tc_workspace_bytes(B, H, T, d_k, d_v, C, 1);
}

int gdn2_chunk_fwd_path(int B, int H, int T, int d_k, int d_v, int C, int dtype) {
    if (B < 0 || H < 0 || T < 0) return 0;
    return select_path(B, H, T, d_k, d_v, C, dtype);
}

int gdn2_chunk_fwd(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
                   const float *S0, void *o, float *S_T, int B, int H, int T, int d_k, int d_v, int C, int dtype,
                   void *workspace, size_t workspace_bytes, void *stream) {
    if (T < 0) return GDN2_ERR_SHAPE;
    int rc;
    if (T == 0) {
        // no tokens: token and output pointers are not read (empty tensors may be NULL)
        if (B < 0 || H < 0) return GDN2_ERR_SHAPE;
        if (dtype != GDN2_F32 && dtype != GDN2_BF16) return GDN2_ERR_DTYPE;
        if (!dim_ok(d_k) || !dim_ok(d_v)) return GDN2_ERR_UNSUPPORTED;
    } else {
        rc = check_common(q, k, v, alpha, b, w, o, B, H, d_k, d_v, dtype);
        if (rc != GDN2_OK) return rc;
    }
    if (C != 64) return GDN2_ERR_UNSUPPORTED;
    if (!S_T) return GDN2_ERR_NULL;
    if (!aligned16(S_T) || (S0 && !aligned16(S0))) return GDN2_ERR_ALIGN;
    if (!workspace) return GDN2_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GDN2_ERR_ALIGN;
    if (workspace_bytes < gdn2_chunk_fwd_workspace_bytes(B, H, T, d_k, d_v, C, dtype)) return GDN2_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (B == 0 || H == 0) return GDN2_OK;
    const size_t state_bytes = sizeof(float) * (size_t)B * H * d_k * d_v;
    if (T == 0) {
        cudaError_t e = S0 ? (S0 == S_T ? cudaSuccess
                                        : cudaMemcpyAsync(S_T, S0, state_bytes, cudaMemcpyDeviceToDevice, st))
                           : cudaMemsetAsync(S_T, 0, state_bytes, st);
        return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
    }
    const int bf16 = dtype == GDN2_BF16 ? 1 : 0;
    const int path = select_path(B, H, T, d_k, d_v, C, dtype);
    if (path == 2)
        rc = gdn2::launch_chunk_split(q, k, v, alpha, b, w, S0, o, S_T, B, H, T, workspace, st);
    else if (path == 1)
        rc = gdn2::launch_chunk_tc(q, k, v, alpha, b, w, S0, o, S_T, B, H, T, d_k, d_v, C, workspace, st);
    else
        rc = gdn2::launch_chunk_simt(q, k, v, alpha, b, w, S0, o, S_T, B, H, T, d_k, d_v, C, bf16, workspace, st);
    return rc;
}

int gdn2_chunk_fwd_edges(const void *q_raw, const void *k_raw, const void *v, const float *a_logit,
                         const void *b_logit, const void *w_logit, const float *S0, const float *o_weight, void *o,
                         float *S_T, int B, int H, int T, int d_k, int d_v, int C, int dtype, void *workspace,
                         size_t workspace_bytes, void *stream) {
    if (T < 0) return GDN2_ERR_SHAPE;
    if (T == 0) return gdn2_chunk_fwd(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, S0, nullptr, S_T, B, H,
                                      0, d_k, d_v, C, dtype, workspace, workspace_bytes, stream);
    int rc = check_common(q_raw, k_raw, v, a_logit, b_logit, w_logit, o, B, H, d_k, d_v, dtype);
    if (rc != GDN2_OK) return rc;
    if (C != 64 || !use_tc(B, H, T, d_k, d_v, C, dtype)) return GDN2_ERR_UNSUPPORTED;
    if (!S_T) return GDN2_ERR_NULL;
    if (!aligned16(S_T) || (S0 && !aligned16(S0)) || (o_weight && !aligned16(o_weight))) return GDN2_ERR_ALIGN;
    if (!workspace) return GDN2_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GDN2_ERR_ALIGN;
    if (workspace_bytes < gdn2_chunk_fwd_edges_workspace_bytes(B, H, T, d_k, d_v, C)) return GDN2_ERR_WORKSPACE;
    if (B == 0 || H == 0) return GDN2_OK;
    if (select_path(B, H, T, d_k, d_v, C, dtype) == 2)
        return gdn2::launch_chunk_split(q_raw, k_raw, v, a_logit, b_logit, w_logit, S0, o, S_T, B, H, T, workspace,
                                        reinterpret_cast<cudaStream_t>(stream), 1, o_weight);
    return gdn2::launch_chunk_tc(q_raw, k_raw, v, a_logit, b_logit, w_logit, S0, o, S_T, B, H, T, d_k, d_v, C,
                                 workspace, reinterpret_cast<cudaStream_t>(stream), 1, o_weight);
}

int gdn2_decode_step(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
                     float *S, void *o, int B, int H, int d_k, int d_v, int dtype, void *stream) {
    int rc = check_common(q, k, v, alpha, b, w, o, B, H, d_k, d_v, dtype);
    if (rc != GDN2_OK) return rc;
    if (!S) return GDN2_ERR_NULL;
    if (!aligned16(S)) return GDN2_ERR_ALIGN;
    if (B == 0 || H == 0) return GDN2_OK;
    return gdn2::launch_decode(q, k, v, alpha, b, w, S, o, B, H, d_k, d_v, dtype == GDN2_BF16 ? 1 : 0,
                               reinterpret_cast<cudaStream_t>(stream));
}

size_t gdn2_chunk_bwd_workspace_bytes(int B, int H, int T, int d_k, int d_v) {
    if (B < 0 || H < 0 || T < 0 || !dim_ok(d_k) || !dim_ok(d_v)) return 0;
    return gdn2::bwd_workspace_bytes(B, H, T, d_k, d_v);
}

int gdn2_chunk_bwd(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
                   const float *S0, const void *dO, const float *dS_T, float *dq, float *dk, float *dv,
                   float *dalpha, float *db, float *dw, float *dS0, int B, int H, int T, int d_k, int d_v,
                   int dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (T < 0 || B < 0 || H < 0) return GDN2_ERR_SHAPE;
    if (dtype != GDN2_F32 && dtype != GDN2_BF16) return GDN2_ERR_DTYPE;
    if (!dim_ok(d_k) || !dim_ok(d_v)) return GDN2_ERR_UNSUPPORTED;
    if ((S0 && !aligned16(S0)) || (dS_T && !aligned16(dS_T)) || (dS0 && !aligned16(dS0))) return GDN2_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t state_bytes = sizeof(float) * (size_t)B * H * d_k * d_v;
    if (T == 0) {   // S_T = S0: dS0 = dS_T; no token gradients
        if (!dS0 || B == 0 || H == 0) return GDN2_OK;
        const cudaError_t e = dS_T ? cudaMemcpyAsync(dS0, dS_T, state_bytes, cudaMemcpyDeviceToDevice, st)
                                   : cudaMemsetAsync(dS0, 0, state_bytes, st);
        return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
    }
    int rc = check_common(q, k, v, alpha, b, w, dO, B, H, d_k, d_v, dtype);
    if (rc != GDN2_OK) return rc;
    if (!dq || !dk || !dv || !dalpha || !db || !dw) return GDN2_ERR_NULL;
    if (!aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(dalpha) || !aligned16(db) ||
        !aligned16(dw))
        return GDN2_ERR_ALIGN;
    if (!workspace) return GDN2_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GDN2_ERR_ALIGN;
    if (workspace_bytes < gdn2_chunk_bwd_workspace_bytes(B, H, T, d_k, d_v)) return GDN2_ERR_WORKSPACE;
    if (B == 0 || H == 0) return GDN2_OK;
    return gdn2::launch_chunk_bwd(q, k, v, alpha, b, w, S0, dO, dS_T, dq, dk, dv, dalpha, db, dw, dS0, B, H, T,
                                  d_k, d_v, dtype == GDN2_BF16 ? 1 : 0, workspace, st);
}

size_t gdn2_chunk_bwd_tc_workspace_bytes(int B, int H, int T, int d_k, int d_v) {
    if (B < 0 || H < 0 || T < 0 || d_k != 128 || d_v != 128) return 0;
    return gdn2::chunk_bwd_tc_workspace_bytes(B, H, T);
}

int gdn2_chunk_bwd_tc(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
                      const float *S0, const void *dO, const float *dS_T, float *dq, float *dk, float *dv,
                      float *dalpha, float *db, float *dw, float *dS0, int B, int H, int T, int d_k, int d_v,
                      int dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (T < 0 || B < 0 || H < 0) return GDN2_ERR_SHAPE;
    if (dtype != GDN2_F32 && dtype != GDN2_BF16) return GDN2_ERR_DTYPE;
    if (dtype != GDN2_BF16 || d_k != 128 || d_v != 128) return GDN2_ERR_UNSUPPORTED;
    if ((S0 && !aligned16(S0)) || (dS_T && !aligned16(dS_T)) || (dS0 && !aligned16(dS0))) return GDN2_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {   // S_T = S0: dS0 = dS_T; no token gradients
        if (!dS0 || B == 0 || H == 0) return GDN2_OK;
        const size_t state_bytes = sizeof(float) * (size_t)B * H * d_k * d_v;
        const cudaError_t e = dS_T ? cudaMemcpyAsync(dS0, dS_T, state_bytes, cudaMemcpyDeviceToDevice, st)
                                   : cudaMemsetAsync(dS0, 0, state_bytes, st);
        return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
    }
    int rc = check_common(q, k, v, alpha, b, w, dO, B, H, d_k, d_v, dtype);
    if (rc != GDN2_OK) return rc;
    if (!dq || !dk || !dv || !dalpha || !db || !dw) return GDN2_ERR_NULL;
    if (!aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(dalpha) || !aligned16(db) ||
        !aligned16(dw))
        return GDN2_ERR_ALIGN;
    if (!workspace) return GDN2_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GDN2_ERR_ALIGN;
    if (workspace_bytes < gdn2_chunk_bwd_tc_workspace_bytes(B, H, T, d_k, d_v)) return GDN2_ERR_WORKSPACE;
    if (B == 0 || H == 0) return GDN2_OK;
    return gdn2::launch_chunk_bwd_tc(q, k, v, alpha, b, w, S0, dO, dS_T, dq, dk, dv, dalpha, db, dw, dS0, B, H, T,
                                     workspace, st);
}

int gdn2_layer_edge_maps(const void *q_raw, const void *k_raw, const float *a_logit, const void *b_logit,
                         const void *w_logit, void *q, void *k, float *alpha, void *b, void *w, int B, int T, int H,
                         int d_k, int d_v, void *stream) {
    if (B < 0 || T < 0 || H < 0) return GDN2_ERR_SHAPE;
    if (!dim_ok(d_k) || !dim_ok(d_v)) return GDN2_ERR_UNSUPPORTED;
    const long long rows = (long long)B * T * H;
    if (rows == 0) return GDN2_OK;
    const void *ptrs[10] = {q_raw, k_raw, a_logit, b_logit, w_logit, q, k, alpha, b, w};
    for (const void *p : ptrs) {
        if (!p) return GDN2_ERR_NULL;
        if (!aligned16(p)) return GDN2_ERR_ALIGN;
    }
    return gdn2::launch_edge_maps(q_raw, k_raw, a_logit, b_logit, w_logit, q, k, alpha, b, w, rows, d_k, d_v,
                                  reinterpret_cast<cudaStream_t>(stream));
}

int gdn2_rms_norm(void *o, const float *weight, long long rows, int d_v, void *stream) {
    if (rows < 0) return GDN2_ERR_SHAPE;
    if (!dim_ok(d_v)) return GDN2_ERR_UNSUPPORTED;
    if (rows == 0) return GDN2_OK;
    if (!o || !weight) return GDN2_ERR_NULL;
    if (!aligned16(o) || !aligned16(weight)) return GDN2_ERR_ALIGN;
    return gdn2::launch_rms_norm(o, weight, rows, d_v, reinterpret_cast<cudaStream_t>(stream));
}

size_t gdn2_gated_norm_bwd_workspace_bytes(long long rows, int d_v) {
    if (rows < 0 || !dim_ok(d_v)) return 0;
    return gdn2::gated_norm_bwd_workspace_bytes(rows, d_v);
}

int gdn2_gated_norm_fwd(const void *o, const void *gate, const float *weight, void *y, long long rows, int d_v, int act,
                        float eps, int dtype, void *stream) {
    int rc = check_norm(rows, eps, dtype);
    if (rc != GDN2_OK) return rc;
    if (act != GDN2_GATE_SILU && act != GDN2_GATE_SIGMOID) return GDN2_ERR_VALUE;
    if (!dim_ok(d_v)) return GDN2_ERR_UNSUPPORTED;
    if (rows == 0) return GDN2_OK;
    if ((rc = check_ptrs({o, gate, weight, y})) != GDN2_OK) return rc;
    return gdn2::launch_gated_norm_fwd(o, gate, weight, y, rows, d_v, act, eps, dtype == GDN2_BF16 ? 1 : 0,
                                       reinterpret_cast<cudaStream_t>(stream));
}

int gdn2_gated_norm_bwd(const void *o, const void *gate, const float *weight, const void *dy, void *d_o, void *dgate,
                        float *dweight, long long rows, int d_v, int act, float eps, int dtype, void *workspace,
                        size_t workspace_bytes, void *stream) {
    int rc = check_norm(rows, eps, dtype);
    if (rc != GDN2_OK) return rc;
    if (act != GDN2_GATE_SILU && act != GDN2_GATE_SIGMOID) return GDN2_ERR_VALUE;
    if (!dim_ok(d_v)) return GDN2_ERR_UNSUPPORTED;
    if (rows > 0 && (rc = check_ptrs({o, gate, dy, d_o, dgate})) != GDN2_OK) return rc;
    if ((rc = check_ptrs({weight, dweight})) != GDN2_OK) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, gdn2::gated_norm_bwd_workspace_bytes(rows, d_v))) != GDN2_OK)
        return rc;
    return gdn2::launch_gated_norm_bwd(o, gate, weight, dy, d_o, dgate, dweight, rows, d_v, act, eps,
                                       dtype == GDN2_BF16 ? 1 : 0, workspace, reinterpret_cast<cudaStream_t>(stream));
}

size_t gdn2_add_norm_bwd_workspace_bytes(long long rows, int width) {
    if (rows < 0 || !width_ok(width)) return 0;
    return gdn2::add_norm_bwd_workspace_bytes(rows, width);
}

int gdn2_add_norm_fwd(const void *x, const void *residual, const float *scale, const float *weight, void *h, void *y,
                      long long rows, int width, float eps, int dtype, void *stream) {
    int rc = check_norm(rows, eps, dtype);
    if (rc != GDN2_OK) return rc;
    if (!width_ok(width)) return GDN2_ERR_UNSUPPORTED;
    if (rows == 0) return GDN2_OK;
    if ((rc = check_ptrs({x, weight, y})) != GDN2_OK) return rc;
    if (!aligned16(residual) || !aligned16(scale) || !aligned16(h)) return GDN2_ERR_ALIGN;   // NULL is aligned
    return gdn2::launch_add_norm_fwd(x, residual, scale, weight, h, y, rows, width, eps, dtype == GDN2_BF16 ? 1 : 0,
                                     reinterpret_cast<cudaStream_t>(stream));
}

int gdn2_add_norm_bwd(const void *h, const void *x, const float *scale, const float *weight, const void *dy,
                      const void *dh, void *dresidual, void *dx, float *dscale, float *dweight, long long rows,
                      int width, float eps, int dtype, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_norm(rows, eps, dtype);
    if (rc != GDN2_OK) return rc;
    if (!width_ok(width)) return GDN2_ERR_UNSUPPORTED;
    if (rows > 0 && (rc = check_ptrs({h, dy, dresidual})) != GDN2_OK) return rc;
    if (rows > 0 && scale && (rc = check_ptrs({x, dx})) != GDN2_OK) return rc;
    if ((rc = check_ptrs({weight, dweight})) != GDN2_OK) return rc;
    if (scale && (rc = check_ptrs({scale, dscale})) != GDN2_OK) return rc;
    if (!aligned16(dh)) return GDN2_ERR_ALIGN;
    if ((rc = check_workspace(workspace, workspace_bytes, gdn2::add_norm_bwd_workspace_bytes(rows, width))) != GDN2_OK)
        return rc;
    return gdn2::launch_add_norm_bwd(h, x, scale, weight, dy, dh, dresidual, dx, dscale, dweight, rows, width, eps,
                                     dtype == GDN2_BF16 ? 1 : 0, workspace, reinterpret_cast<cudaStream_t>(stream));
}

int gdn2_tree_fwd(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
                  const float *S, long long slot_stride, int num_slots, const int *slots, const int *cu_nodes,
                  const int *parents, void *o, int batch, int H, int total, int max_nodes, int d_k, int d_v, int dtype,
                  void *workspace, size_t workspace_bytes, void *stream) {
    if (batch < 0 || total < 0 || max_nodes < 0 || num_slots < 0) return GDN2_ERR_SHAPE;
    if (total == 0) {   // empty token tensors may be NULL
        if (H < 0) return GDN2_ERR_SHAPE;
        if (dtype != GDN2_F32 && dtype != GDN2_BF16) return GDN2_ERR_DTYPE;
        if (!dim_ok(d_k) || !dim_ok(d_v)) return GDN2_ERR_UNSUPPORTED;
    } else {
        const int rc = check_common(q, k, v, alpha, b, w, o, batch, H, d_k, d_v, dtype);
        if (rc != GDN2_OK) return rc;
    }
    if (max_nodes > GDN2_TREE_MAX_NODES || batch > 65535) return GDN2_ERR_UNSUPPORTED;
    int rc = check_pool(S, slot_stride, num_slots, H, d_k, d_v);
    if (rc != GDN2_OK) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, gdn2::kStatusBytes)) != GDN2_OK) return rc;
    if (batch == 0 || H == 0 || total == 0 || max_nodes == 0) return GDN2_OK;
    if (!slots || !cu_nodes || !parents) return GDN2_ERR_NULL;
    if (!aligned4(slots) || !aligned4(cu_nodes) || !aligned4(parents)) return GDN2_ERR_ALIGN;
    return gdn2::launch_tree(q, k, v, alpha, b, w, S, slot_stride, num_slots, slots, cu_nodes, parents, o, batch, H,
                             total, max_nodes, d_k, d_v, dtype == GDN2_BF16 ? 1 : 0,
                             reinterpret_cast<unsigned *>(workspace), reinterpret_cast<cudaStream_t>(stream));
}

int gdn2_recurrent_fwd(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
                       float *S, long long slot_stride, int num_slots, const int *slots_in, const int *slots_out,
                       const int *cu_tokens, const int *index, void *o, int batch, int H, int total, int rows, int d_k,
                       int d_v, int dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (batch < 0 || total < 0 || rows < 0 || num_slots < 0) return GDN2_ERR_SHAPE;
    if (!index && total > rows) return GDN2_ERR_SHAPE;
    if (total == 0) {   // no tokens: states are copied or cleared, token tensors may be NULL
        if (H < 0) return GDN2_ERR_SHAPE;
        if (dtype != GDN2_F32 && dtype != GDN2_BF16) return GDN2_ERR_DTYPE;
        if (!dim_ok(d_k) || !dim_ok(d_v)) return GDN2_ERR_UNSUPPORTED;
    } else {
        // o is optional: without it only the states are advanced
        const int rc = check_common(q, k, v, alpha, b, w, o ? o : q, batch, H, d_k, d_v, dtype);
        if (rc != GDN2_OK) return rc;
    }
    if (batch > 65535 || H > 65535) return GDN2_ERR_UNSUPPORTED;
    int rc = check_pool(S, slot_stride, num_slots, H, d_k, d_v);
    if (rc != GDN2_OK) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, gdn2::kStatusBytes)) != GDN2_OK) return rc;
    if (batch == 0 || H == 0) return GDN2_OK;
    if (!slots_in || !slots_out || !cu_tokens) return GDN2_ERR_NULL;
    if (!aligned4(slots_in) || !aligned4(slots_out) || !aligned4(cu_tokens) || !aligned4(index)) return GDN2_ERR_ALIGN;
    return gdn2::launch_recurrent(q, k, v, alpha, b, w, S, slot_stride, num_slots, slots_in, slots_out, cu_tokens,
                                  index, o, batch, H, total, rows, d_k, d_v, dtype == GDN2_BF16 ? 1 : 0,
                                  reinterpret_cast<unsigned *>(workspace), reinterpret_cast<cudaStream_t>(stream));
}

int gdn2_state_copy(float *dst, long long dst_stride, int dst_slots, const float *src, long long src_stride,
                    int src_slots, const int *dst_index, const int *src_index, int pairs, long long slot_floats,
                    void *workspace, size_t workspace_bytes, void *stream) {
    if (dst_slots < 0 || src_slots < 0 || pairs < 0 || slot_floats < 0) return GDN2_ERR_SHAPE;
    if (dst_stride < slot_floats || src_stride < slot_floats) return GDN2_ERR_SHAPE;
    if (slot_floats % 4 || dst_stride % 4 || src_stride % 4) return GDN2_ERR_ALIGN;
    if (pairs > GDN2_STATE_COPY_MAX_PAIRS || slot_floats > (1ll << 31)) return GDN2_ERR_UNSUPPORTED;
    if (dst == src && dst_slots > 1 && src_slots > 1 && dst_stride != src_stride) return GDN2_ERR_SHAPE;
    if (caches_clash(dst, dst_stride, dst_slots, src, src_stride, src_slots, slot_floats)) return GDN2_ERR_SHAPE;
    int rc = check_workspace(workspace, workspace_bytes, gdn2::kStatusBytes);
    if (rc != GDN2_OK) return rc;
    if (pairs == 0 || slot_floats == 0) return GDN2_OK;
    if ((dst_slots && !dst) || (src_slots && !src) || !dst_index || !src_index) return GDN2_ERR_NULL;
    if (!aligned16(dst) || !aligned16(src) || !aligned4(dst_index) || !aligned4(src_index)) return GDN2_ERR_ALIGN;
    return gdn2::launch_state_copy(dst, dst_stride, dst_slots, src, src_stride, src_slots, dst_index, src_index, pairs,
                                   slot_floats, reinterpret_cast<unsigned *>(workspace),
                                   reinterpret_cast<cudaStream_t>(stream));
}

int gdn2_gemm_phase_probe(int mode, int reps, int nctas, void *workspace, size_t workspace_bytes, void *stream) {
    if ((mode != 0 && mode != 1) || reps < 1 || nctas < 1) return GDN2_ERR_SHAPE;
    if (!workspace) return GDN2_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GDN2_ERR_ALIGN;
    if (workspace_bytes < gdn2::kStatusBytes) return GDN2_ERR_WORKSPACE;
    return gdn2::launch_phase_probe(mode, reps, nctas, reinterpret_cast<unsigned int *>(workspace),
                                    reinterpret_cast<cudaStream_t>(stream));
}

int gdn2_set_wait_limit(long long polls) {
    if (polls < -1 || polls > 0xffffffffll) return GDN2_ERR_VALUE;
    t_wait_limit = polls;
    return GDN2_OK;
}

int gdn2_workspace_status(void *workspace, int clear, int *out, void *stream) {
    if (!workspace || !out) return GDN2_ERR_NULL;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    unsigned int word = 0;
    if (cudaMemcpyAsync(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost, st) != cudaSuccess)
        return GDN2_ERR_CUDA;
    if (cudaStreamSynchronize(st) != cudaSuccess) return GDN2_ERR_CUDA;
    *out = (int)word;
    if (clear && word) {
        if (cudaMemsetAsync(workspace, 0, gdn2::kStatusBytes, st) != cudaSuccess) return GDN2_ERR_CUDA;
        if (cudaStreamSynchronize(st) != cudaSuccess) return GDN2_ERR_CUDA;
    }
    return GDN2_OK;
}

const char *gdn2_status_str(int status) {
    switch (status) {
        case GDN2_OK: return "ok";
        case GDN2_ERR_NULL: return "a required pointer is NULL";
        case GDN2_ERR_SHAPE: return "a size is negative or inconsistent";
        case GDN2_ERR_DTYPE: return "unknown dtype code";
        case GDN2_ERR_UNSUPPORTED: return "unsupported size (d_k and d_v must be 64 or 128, C must be 64)";
        case GDN2_ERR_WORKSPACE: return "workspace missing or too small";
        case GDN2_ERR_CUDA: return "CUDA runtime or launch error";
        case GDN2_ERR_ALIGN: return "a pointer is not 16-byte aligned";
        case GDN2_ERR_DEVICE: return "a kernel reported an internal error";
        case GDN2_ERR_NOALLOC_LIMIT:
            return "problem needs more scratch than the no-allocation entry point's fixed array";
        case GDN2_ERR_VALUE: return "an argument's value is out of its range";
        default: return "unknown status";
    }
}

}  // extern "C"
