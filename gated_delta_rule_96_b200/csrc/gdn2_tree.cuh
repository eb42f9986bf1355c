// What the two kernels for drafted trees share (sm_100a): paths to the root and the coefficients along them.
#pragma once

#include "gdn2_internal.h"
#include "gdn2_slots.cuh"

namespace gdn2 {
namespace tree {

constexpr int MAX_NODES = kTreeMaxNodes;

// The tensor-core kernel (bf16 tokens, d_k = d_v = 128), gdn2_tree_tc.cu.
int launch_tc(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
              const float *S, long long slot_stride, int num_slots, const int *slots, const int *cu, const int *parents,
              void *o, int batch, int H, int total, int max_nodes, unsigned *status, cudaStream_t st);

// A node's row of coefficients starts at pairs(node): for itself, then its parent, and on to its root, at most
// node + 1 in all, filled up to a multiple of four (zeros, for the root).
__host__ __device__ constexpr int pairs(int node) { return 4 * (node / 4 + 1) * (2 * (node / 4) + node % 4); }
constexpr int MAX_PAIRS = pairs(MAX_NODES);
static_assert(pairs(0) == 0 && pairs(1) == 4 && pairs(4) == 16 && pairs(5) == 24 && pairs(64) == 2176, "row starts");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// What follows the paths takes eight lanes a node, four nodes a warp; all lanes of a warp make the calls, and
// `go` says whether the lane's node takes part (its eight lanes alike).

// One thread lists the path from a node to its root; the number of ancestors is returned.
template <typename Parent>
__device__ __forceinline__ int list_path(const Parent *parent, unsigned char *anc, int node) {
    int out = pairs(node), at = node, above = -1;
    for (int up = node; up >= 0; up = parent[up]) {
        at = up;
        anc[out++] = (unsigned char)at;
        ++above;
    }
    while (out & 3) anc[out++] = (unsigned char)at;   // behind the root: the root again
    return above;
}

// Whether G_n and 1 / G_n can stand for themselves: at all the node's channels in [2^-80, 2^80], far enough from the
// ends of fp32 for the products with tokens and for the second of two bf16 parts.
template <int K>
__device__ __forceinline__ bool in_range(const f32x2 (&G)[K / 32][2], int lane) {
    bool fine = true;
#pragma unroll
    for (int j = 0; j < K / 32; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float2 x = unpack2(G[j][c]);
            fine = fine && x.x >= 0x1p-80f && x.x <= 0x1p80f && x.y >= 0x1p-80f && x.y <= 0x1p80f;   // false for a NaN
        }
    return (__ballot_sync(0xffffffffu, fine) >> (lane & 24) & 0xffu) == 0xffu;
}

// A and P of a node's path, to cA and cP, with the decays multiplied in one by one on the way up, from the tokens in
// HBM: for decays whose product leaves the range (zero among them), exact for any.
template <typename Tok, int K>
__device__ __forceinline__ void couple_far(const Tok *q, const Tok *k, const Tok *b, const float *alpha,
                                        const unsigned char *anc, float *cA, float *cP, bool go, int lo, int H, int head,
                                        int node, int above, int lane) {
    const int sub = lane & 7, base = pairs(go ? node : 0), most = __reduce_max_sync(0xffffffffu, go ? above : -1);
    const auto row = [&](int i) { return ((size_t)(lo + i) * H + head) * K + 4 * sub; };
    float e[K / 32][4], g[K / 32][4];
#pragma unroll
    for (int j = 0; j < K / 32; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const size_t at = row(go ? node : 0) + 32 * j + c;
            e[j][c] = ld_tok(b + at) * ld_tok(k + at);
            g[j][c] = ld_tok(q + at);
        }
    for (int i = 0; i <= most; ++i) {
        const bool some = go && i <= above;
        const size_t at = row(some ? anc[base + i] : 0);
        float a = 0.f, p = 0.f;
#pragma unroll
        for (int j = 0; j < K / 32; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float kk = ld_tok(k + at + 32 * j + c), aa = alpha[at + 32 * j + c];
                a = fmaf(e[j][c], kk, a);
                p = fmaf(g[j][c], kk, p);
                e[j][c] *= aa;
                g[j][c] *= aa;
            }
#pragma unroll
        for (int m = 4; m > 0; m >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, m);
            p += __shfl_xor_sync(0xffffffffu, p, m);
        }
        if (some && sub == 0) cA[base + i] = a, cP[base + i] = p;
    }
}

// The deltas eliminated: with p_0 = n, p_1, ... the path from n to its root and R[i] = u_i - S^T (e_i G_i),
//   o_n = S^T (q_n G_n) + sum_j C[n,j] R[p_j],   C[n,j] = P[n,p_j] - sum_{m < j} C[n,m] A[p_m, p_j]
// A node's C needs no other node's, so the columns' work has no order among the nodes left: one product for
// each pair, in place of two and a barrier for each level of the tree.  Lane `sub` takes j = 8 h + sub; the
// coefficients of a finished j go to the others by a shuffle, those of finished blocks of eight through
// shared memory.  The A and P of all nodes must be there; cC may be cP.
__device__ __forceinline__ void eliminate(const float *cA, const float *cP, const unsigned char *anc, float *cC, bool go,
                                          int node, int above, int lane) {
    const int sub = lane & 7, team = lane & 24, base = pairs(go ? node : 0);
    if (!go) above = -1;
    const int most = __reduce_max_sync(0xffffffffu, above);
    const auto row = [&](int j) { return j <= above ? pairs(anc[base + j]) : 0; };   // of an ancestor's own A
#pragma unroll 1
    for (int h = 0; h <= most; h += 8) {
        const int j = h + sub;
        const bool mine = j <= above;
        float c = mine ? cP[base + j] : 0.f, up[8];
        const int start = row(j);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            const int from = __shfl_sync(0xffffffffu, start, team | m);
            up[m] = mine && m < sub ? cA[from + sub - m] : 0.f;
        }
#pragma unroll 1
        for (int f = 0; f < h; f += 8) {   // finished blocks
            const int first = row(f + sub);
            const float done = f + sub <= above ? cC[base + f + sub] : 0.f;
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                const int from = __shfl_sync(0xffffffffu, first, team | m);
                const float x = __shfl_sync(0xffffffffu, done, team | m);
                if (mine) c = fmaf(-x, cA[from + j - f - m], c);
            }
        }
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            const float done = __shfl_sync(0xffffffffu, c, team | m);
            if (m < sub) c = fmaf(-done, up[m], c);
        }
        if (j <= (above | 3)) cC[base + j] = mine ? c : 0.f;   // with the zeros that fill the row up
        __syncwarp();
    }
}

}  // namespace tree
}  // namespace gdn2
