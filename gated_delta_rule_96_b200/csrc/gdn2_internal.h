// Host-side launchers shared between the ABI layer and the kernel files.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn2 {

// Whether a runtime call succeeded.  One that did not is reported by the call at hand; its error does not stay behind
// for the next one that asks for the last error.
inline bool succeeded(cudaError_t e) {
    if (e == cudaSuccess) return true;
    cudaGetLastError();
    return false;
}

// Lets `kern` use up to `bytes` of dynamic shared memory on the current device.  At every launch, since the
// attribute is a device's (and a context's) own and setting it takes a fraction of a microsecond; always the most
// that any launch of the kernel uses, since another host thread may be between this and its launch.
template <typename Kernel>
inline bool allow_smem(Kernel kern, size_t bytes) {
    return succeeded(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
}

// A launch that the device prepares while the stream's kernel before it still runs: its blocks are placed as that
// one's leave, and wait there for its end.  One call behind another, us, without and with it: a fork 5.6 / 3.2, one
// user's tree 8.8 / 6.8, a decode step of residual norms 5.4 / 4.9 (the host), B256 H16 of runs 102 / 99 (each as the kernel was then).
// (griddepcontrol.launch_dependents at the top of every kernel, which lets the next one's blocks in as soon as all of
// its own have started, is slower: 3.5, 7.0, 4.8, 100, and the full batch of trees 142 against 137.)
template <typename... Params, typename... Args>
inline int launch_close(void (*kern)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchAttribute close = {};
    close.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    close.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = grid;
    config.blockDim = dim3((unsigned)threads);
    config.dynamicSmemBytes = smem;
    config.stream = st;
    config.attrs = &close;
    config.numAttrs = 1;
    return succeeded(cudaLaunchKernelEx(&config, kern, static_cast<Params>(args)...)) ? 0 : -6;
}
// In every such kernel, before any access to memory that is not the block's own: waits until the kernel before
// has ended and its writes can be seen.
__device__ __forceinline__ void behind_last_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Polls of a bounded wait in the next launch: `usual`, unless the calling thread has set another limit
// (gdn2_set_wait_limit).
uint32_t wait_limit(uint32_t usual);

// Status header at the start of every prefill workspace (device status words).
constexpr size_t kStatusBytes = 256;

// Decode: one token per (b, h); S updated in place.
int launch_decode(const void *q, const void *k, const void *v, const float *alpha, const void *b,
                  const void *w, float *S, void *o, int B, int H, int K, int V, int bf16, cudaStream_t st);

// SIMT two-kernel prefill (fp32 FMA everywhere; any token dtype).
size_t simt_workspace_bytes(int B, int H, int T, int K, int V, int C);
int launch_chunk_simt(const void *q, const void *k, const void *v, const float *alpha, const void *b,
                      const void *w, const float *S0, void *o, float *ST, int B, int H, int T, int K, int V,
                      int C, int bf16, void *ws, cudaStream_t st);

// Fused tcgen05 prefill (bf16 tokens, d_k = d_v = 128, C = 64).
bool tc_supported(int B, int H, int T, int K, int V, int C, int bf16);
// edges != 0: the layer-edge variant's ring (RING_SLOTS x 80 KB per block) is included
size_t tc_workspace_bytes(int B, int H, int T, int K, int V, int C, int edges = 0);
// edges != 0: q, k, b, w, alpha are the layer's raw inputs (see gdn2_chunk_fwd_edges); onorm, if
// not null, is the RMSNorm weight applied to o.
int launch_chunk_tc(const void *q, const void *k, const void *v, const float *alpha, const void *b,
                    const void *w, const float *S0, void *o, float *ST, int B, int H, int T, int K, int V,
                    int C, void *ws, cudaStream_t st, int edges = 0, const float *onorm = nullptr);

// Two-stage tcgen05 prefill (bf16 tokens, d_k = d_v = 128, C = 64): the intra-chunk work in parallel
// over every chunk-head, then the state chain; long sequences in windows, few long chains cut into
// segments in time.
size_t split_workspace_bytes(int B, int H, int T);
// edges != 0: q, k, b, w, alpha are the layer's raw inputs (see gdn2_chunk_fwd_edges); onorm, if not
// null, is the RMSNorm weight applied to o.
int launch_chunk_split(const void *q, const void *k, const void *v, const float *alpha, const void *b,
                       const void *w, const float *S0, void *o, float *ST, int B, int H, int T, void *ws,
                       cudaStream_t st, int edges = 0, const float *onorm = nullptr);

// Measurement kernel of the prefill's tensor-core phases (mode 0: back to back; 1: each group waits
// for the previous one), `reps` chunks per CTA on `nctas` CTAs.
int launch_phase_probe(int mode, int reps, int nctas, unsigned int *status, cudaStream_t st);

// S_g = M_(g-1) S_(g-1) + N_(g-1) along nseg segments of each chain (fp32; M, N, Sg [chains][nseg][128][128],
// S0 [chains][128][128] or null for zero).
int launch_segment_scan(const float *M, const float *N, const float *S0, float *Sg, int chains, int nseg,
                        cudaStream_t st);

// The layer's edge maps on their own (bf16 tokens, d in {64, 128}; rows = B*T*H).
int launch_edge_maps(const void *q_raw, const void *k_raw, const float *a_logit, const void *b_logit,
                     const void *w_logit, void *q, void *k, float *alpha, void *b, void *w, long long rows, int K, int V,
                     cudaStream_t st);
int launch_rms_norm(void *o, const float *weight, long long rows, int V, cudaStream_t st);

// Backward pass (three sequential passes per chain; fp32 gradients; d_k, d_v in {64, 128}).
size_t bwd_workspace_bytes(int B, int H, int T, int K, int V);
int launch_chunk_bwd(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
                     const float *S0, const void *dO, const float *dST, float *dq, float *dk, float *dv,
                     float *dalpha, float *db, float *dw, float *dS0, int B, int H, int T, int K, int V, int bf16,
                     void *ws, cudaStream_t st);

// Tensor-core backward (bf16 tokens, d_k = d_v = 128): forward replay by the two-stage prefill's kernels,
// reverse walk of the state gradient, gradient kernel over every chunk-head.
size_t chunk_bwd_tc_workspace_bytes(int B, int H, int T);
int launch_chunk_bwd_tc(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
                        const float *S0, const void *dO, const float *dST, float *dq, float *dk, float *dv,
                        float *dalpha, float *db, float *dw, float *dS0, int B, int H, int T, void *ws,
                        cudaStream_t st);

// The layer's norms with their gradients (d_v in {64, 128}; width a multiple of 8, at most 8192).
size_t gated_norm_bwd_workspace_bytes(long long rows, int D);
size_t add_norm_bwd_workspace_bytes(long long rows, int width);
int launch_gated_norm_fwd(const void *o, const void *gate, const float *weight, void *y, long long rows, int D, int act,
                          float eps, int bf16, cudaStream_t st);
int launch_gated_norm_bwd(const void *o, const void *gate, const float *weight, const void *dy, void *d_o, void *dgate,
                          float *dweight, long long rows, int D, int act, float eps, int bf16, void *ws,
                          cudaStream_t st);
int launch_add_norm_fwd(const void *x, const void *residual, const float *scale, const float *weight, void *h, void *y,
                        long long rows, int width, float eps, int bf16, cudaStream_t st);
int launch_add_norm_bwd(const void *h, const void *x, const float *scale, const float *weight, const void *dy,
                        const void *dh, void *dres, void *dx, float *dscale, float *dweight, long long rows, int width,
                        float eps, int bf16, void *ws, cudaStream_t st);

// Over slots of a state cache: drafted trees, ragged runs, copies (d_k, d_v in {64, 128}).
constexpr int kTreeMaxNodes = 64;
constexpr int kStateCopyMaxPairs = 1024;
int launch_tree(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
                const float *S, long long slot_stride, int num_slots, const int *slots, const int *cu,
                const int *parents, void *o, int batch, int H, int total, int max_nodes, int K, int V, int bf16,
                unsigned *status, cudaStream_t st);
int launch_recurrent(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
                     float *S, long long slot_stride, int num_slots, const int *slots_in, const int *slots_out,
                     const int *cu, const int *index, void *o, int batch, int H, int total, int rows, int K, int V,
                     int bf16, unsigned *status, cudaStream_t st);
int launch_state_copy(float *dst, long long dst_stride, int dst_slots, const float *src, long long src_stride,
                      int src_slots, const int *dst_idx, const int *src_idx, int n, long long slot_floats,
                      unsigned *status, cudaStream_t st);

}  // namespace gdn2
