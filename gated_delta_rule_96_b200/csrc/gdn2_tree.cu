// Drafted tokens in a tree over a state cache: the read-out of every node, the cache unchanged (sm_100a;
// page "NVIDIA представила Gated DeltaNet-2 ...", section "Техническая схема", the state-update equation, and
// the paragraph on the chunkwise WY form).
//
// A node's state is its parent's after one step of the recurrence; a root's parent is the cached state S.
// With G_n the channel-wise product of the decays on the path from S to n (n's own included), e = b k and
// u = w v, the states need not be formed:
//   delta_n = u_n - S^T (e_n G_n) - sum over proper ancestors i of A[n,i] delta_i,   A[n,i] = sum_c e_n (G_n / G_i) k_i
//   o_n     = S^T (q_n G_n) + sum over ancestors i and n itself of P[n,i] delta_i,   P[n,i] = sum_c q_n (G_n / G_i) k_i
// G_n / G_i is the product of the decays below i down to n, so walking from n to its root with a running
// product gives A, P, e_n G_n and q_n G_n without a division, a logarithm or a masked entry: decays of any
// size (zero included) are exact, and what sits on another branch is never touched.
#include "gdn2_internal.h"
#include "gdn2_slots.cuh"

namespace gdn2 {
namespace tree {

constexpr int MAX_NODES = kTreeMaxNodes;

size_t smem_bytes(int n, int K, int V) {
    return sizeof(float) * ((size_t)n * (4 * K + 2 * V) + 2 * (size_t)n * n) + sizeof(int) * (size_t)MAX_NODES;
}

// One block per (head, sequence), 16 columns of the state a warp (2 V threads).
template <typename Tok, int K, int V>
__global__ void __launch_bounds__(2 * V) tree_kernel(const Tok *__restrict__ q, const Tok *__restrict__ k,
                                                     const Tok *__restrict__ v, const float *__restrict__ alpha,
                                                     const Tok *__restrict__ b, const Tok *__restrict__ w,
                                                     const float *__restrict__ S, long long slot_stride, int num_slots,
                                                     const int *__restrict__ slots, const int *__restrict__ cu,
                                                     const int *__restrict__ parents, Tok *__restrict__ o, int H,
                                                     int total, int max_nodes, unsigned *status) {
    constexpr int RJ = K / 32, NT = 2 * V;
    extern __shared__ __align__(16) float smem[];
    float *sk = smem, *se = sk + max_nodes * K, *sq = se + max_nodes * K, *sa = sq + max_nodes * K;
    float *sr = sa + max_nodes * K, *ss = sr + max_nodes * V, *sA = ss + max_nodes * V, *sP = sA + max_nodes * max_nodes;
    int *sp = reinterpret_cast<int *>(sP + max_nodes * max_nodes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rg = lane & 7, cg = lane >> 3;
    const int head = blockIdx.x, seq = blockIdx.y;

    const int lo = cu[seq], hi = cu[seq + 1], slot = slots[seq];
    unsigned bad = 0;
    if (lo < 0 || hi < lo || hi > total || hi - lo > max_nodes) bad = DEV_RANGE;
    else if (slot < -1 || slot >= num_slots) bad = DEV_SLOT;
    else if (tid < hi - lo) {
        const int p = parents[lo + tid];
        if (p < -1 || p >= tid) bad = DEV_PARENT;
        sp[tid] = p;
    }
    if (__syncthreads_or(bad != 0)) {
        if (bad) atomicOr(status, bad);
        return;
    }
    const int n = hi - lo;
    if (n == 0) return;

    for (int i = tid; i < n * K; i += NT) {
        const size_t at = ((size_t)(lo + i / K) * H + head) * K + i % K;
        const float kk = ld_tok(k + at);
        sk[i] = kk;
        se[i] = ld_tok(b + at) * kk;
        sq[i] = ld_tok(q + at);
        sa[i] = alpha[at];
    }
    // the slice of the state: rows 4 (rg + 8 j) + i, columns c0 .. c0 + 3
    const int c0 = warp * 16 + cg * 4;
    float s[RJ][4][4];
#pragma unroll
    for (int j = 0; j < RJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (slot >= 0)
                x = ld_stream(reinterpret_cast<const float4 *>(S + (size_t)slot * slot_stride + (size_t)head * K * V +
                                                               (size_t)(4 * (rg + 8 * j) + i) * V + c0));
            s[j][i][0] = x.x; s[j][i][1] = x.y; s[j][i][2] = x.z; s[j][i][3] = x.w;
        }
    __syncthreads();

    // A and P: eight lanes a node, from the node to its root
    for (int n0 = warp * 4; n0 < n; n0 += NT / 8) {
        const int node = n0 + cg;
        const bool have = node < n;
        float ek[RJ][4], qk[RJ][4];
        auto row = [&](const float *x, int at, int j) {
            return *reinterpret_cast<const float4 *>(x + at * K + 4 * (rg + 8 * j));
        };
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
            const float4 x = row(se, have ? node : 0, j), y = row(sq, have ? node : 0, j);
            ek[j][0] = x.x; ek[j][1] = x.y; ek[j][2] = x.z; ek[j][3] = x.w;
            qk[j][0] = y.x; qk[j][1] = y.y; qk[j][2] = y.z; qk[j][3] = y.w;
        }
        int at = have ? node : -1;
        while (__any_sync(0xffffffffu, at >= 0)) {
            const int i = at < 0 ? 0 : at;
            float a = 0.f, p = 0.f;
#pragma unroll
            for (int j = 0; j < RJ; ++j) {
                const float4 k4 = row(sk, i, j), a4 = row(sa, i, j);
                const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, aa[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    a = fmaf(ek[j][c], kk[c], a);
                    p = fmaf(qk[j][c], kk[c], p);
                    if (at >= 0) {
                        ek[j][c] *= aa[c];
                        qk[j][c] *= aa[c];
                    }
                }
            }
#pragma unroll
            for (int m = 4; m > 0; m >>= 1) {
                a += __shfl_xor_sync(0xffffffffu, a, m);
                p += __shfl_xor_sync(0xffffffffu, p, m);
            }
            if (at >= 0) {
                if (rg == 0) {
                    sA[node * max_nodes + at] = a;
                    sP[node * max_nodes + at] = p;
                }
                at = sp[at];
            }
        }
        if (have)
#pragma unroll
            for (int j = 0; j < RJ; ++j) {   // e_n G_n and q_n G_n in place: no other node reads this row
                *reinterpret_cast<float4 *>(se + node * K + 4 * (rg + 8 * j)) =
                    make_float4(ek[j][0], ek[j][1], ek[j][2], ek[j][3]);
                *reinterpret_cast<float4 *>(sq + node * K + 4 * (rg + 8 * j)) =
                    make_float4(qk[j][0], qk[j][1], qk[j][2], qk[j][3]);
            }
    }
    __syncthreads();

    // S^T (e G) and S^T (q G) of every node
    for (int t = 0; t < n; ++t) {
        float p[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) p[c] = 0.f;
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
            const float4 e4 = *reinterpret_cast<const float4 *>(se + t * K + 4 * (rg + 8 * j));
            const float4 q4 = *reinterpret_cast<const float4 *>(sq + t * K + 4 * (rg + 8 * j));
            const float ee[4] = {e4.x, e4.y, e4.z, e4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    p[c] = fmaf(ee[i], s[j][i][c], p[c]);
                    p[4 + c] = fmaf(qq[i], s[j][i][c], p[4 + c]);
                }
        }
        const float sum = scatter_sum8(p, lane);
        (rg < 4 ? sr : ss)[t * V + c0 + (rg & 3)] = sum;
    }
    __syncthreads();

    // delta and o, node by node (a parent comes before its children), a column a thread
    if (tid < V)
        for (int t = 0; t < n; ++t) {
            const size_t at = ((size_t)(lo + t) * H + head) * V + tid;
            float d = ld_tok(w + at) * ld_tok(v + at) - sr[t * V + tid], x = ss[t * V + tid];
            for (int i = sp[t]; i >= 0; i = sp[i]) {
                const float di = sr[i * V + tid];
                d = fmaf(-sA[t * max_nodes + i], di, d);
                x = fmaf(sP[t * max_nodes + i], di, x);
            }
            sr[t * V + tid] = d;
            store_tok(o + at, fmaf(sP[t * max_nodes + t], d, x));
        }
}

template <typename Tok, int K, int V>
int launch_t(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
             const float *S, long long slot_stride, int num_slots, const int *slots, const int *cu, const int *parents,
             void *o, int batch, int H, int total, int max_nodes, unsigned *status, cudaStream_t st) {
    const size_t smem = smem_bytes(max_nodes, K, V);
    if (cudaFuncSetAttribute(tree_kernel<Tok, K, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess)
        return -6;
    tree_kernel<Tok, K, V><<<dim3(H, batch), 2 * V, smem, st>>>(
        (const Tok *)q, (const Tok *)k, (const Tok *)v, alpha, (const Tok *)b, (const Tok *)w, S, slot_stride,
        num_slots, slots, cu, parents, (Tok *)o, H, total, max_nodes, status);
    return launch_status();
}

}  // namespace tree

int launch_tree(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
                const float *S, long long slot_stride, int num_slots, const int *slots, const int *cu,
                const int *parents, void *o, int batch, int H, int total, int max_nodes, int K, int V, int bf16,
                unsigned *status, cudaStream_t st) {
    auto go = [&](auto launch) {
        return launch(q, k, v, alpha, b, w, S, slot_stride, num_slots, slots, cu, parents, o, batch, H, total,
                      max_nodes, status, st);
    };
    if (bf16) {
        if (K == 128) return V == 128 ? go(tree::launch_t<__nv_bfloat16, 128, 128>) : go(tree::launch_t<__nv_bfloat16, 128, 64>);
        return V == 128 ? go(tree::launch_t<__nv_bfloat16, 64, 128>) : go(tree::launch_t<__nv_bfloat16, 64, 64>);
    }
    if (K == 128) return V == 128 ? go(tree::launch_t<float, 128, 128>) : go(tree::launch_t<float, 128, 64>);
    return V == 128 ? go(tree::launch_t<float, 64, 128>) : go(tree::launch_t<float, 64, 64>);
}

}  // namespace gdn2
