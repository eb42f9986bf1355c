// What the two kernels for drafted trees share (sm_100a): the walk from a node to its root.
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

// A node's coefficients {A, P} lie at ap[pairs(node)] for itself, then its parent, and on to its root, the node
// that each is for at the same place of anc: a node has at most `node` ancestors, so the rows never meet.
__host__ __device__ constexpr int pairs(int node) { return node * (node + 1) / 2; }

// Eight lanes take one node (four nodes a warp; all lanes of the warp call this, with a node >= n for none) from
// it to its root, 16 or 8 channels each: channels 4 (sub + 8 j) + c, sub = lane & 7.  On return e and g are
// e_n G_n and q_n G_n, and the node's rows of ap and anc are written.  sk, sa: k and alpha of all nodes in
// shared memory; parent: theirs.  Four operations a channel, and shuffles over eight lanes for each pair
// (node, ancestor): the decays are multiplied in as the walk goes up.
template <typename Tok, int K, typename SharedTok, typename Parent>
__device__ __forceinline__ void walk(const Tok *k, const Tok *b, const Tok *q, const SharedTok *sk, const float *sa,
                                     const Parent *parent, float2 *ap, unsigned char *anc, int lo, int H, int head,
                                     int node, int n, int lane, float (&e)[K / 32][4], float (&g)[K / 32][4]) {
    constexpr int RJ = K / 32;
    const int sub = lane & 7;
    const auto key = [&](int at, int j, float (&x)[4]) {
        Raw<SharedTok, 4> r;
        r.load(sk + at * K + 4 * (sub + 8 * j));
        r.get(x);
    };
    int at = node < n ? node : -1;
    {
        Raw<Tok, 4> rb[RJ], rq[RJ];
        const int mine = at < 0 ? 0 : at;
        const size_t row = ((size_t)(lo + mine) * H + head) * K + 4 * sub;
#pragma unroll
        for (int j = 0; j < RJ; ++j) rb[j].load(b + row + 32 * j), rq[j].load(q + row + 32 * j);
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
            float kk[4];
            key(mine, j, kk);
            rb[j].get(e[j]);
            rq[j].get(g[j]);
#pragma unroll
            for (int c = 0; c < 4; ++c) e[j][c] *= kk[c];
        }
    }
    int out = pairs(at < 0 ? 0 : at);
    while (__any_sync(0xffffffffu, at >= 0)) {
        float a = 0.f, p = 0.f;
        if (at >= 0) {
#pragma unroll
            for (int j = 0; j < RJ; ++j) {
                float kk[4];
                key(at, j, kk);
                const float4 a4 = *reinterpret_cast<const float4 *>(sa + at * K + 4 * (sub + 8 * j));
                const float aa[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    a = fmaf(e[j][c], kk[c], a);
                    p = fmaf(g[j][c], kk[c], p);
                    e[j][c] *= aa[c];
                    g[j][c] *= aa[c];
                }
            }
        }
#pragma unroll
        for (int m = 4; m > 0; m >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, m);
            p += __shfl_xor_sync(0xffffffffu, p, m);
        }
        if (at >= 0) {
            if (sub == 0) ap[out] = make_float2(a, p), anc[out] = (unsigned char)at;   // its own A is not used
            ++out;
            at = parent[at];
        }
    }
}

}  // namespace tree
}  // namespace gdn2
