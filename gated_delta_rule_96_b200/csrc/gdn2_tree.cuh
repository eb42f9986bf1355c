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

// A node's row of coefficients starts at pairs(node): for itself, then its parent, and on to its root, at most
// node + 1 in all, filled up to a multiple of four (zeros, for the root).
__host__ __device__ constexpr int pairs(int node) { return 4 * (node / 4 + 1) * (2 * (node / 4) + node % 4); }
constexpr int MAX_PAIRS = pairs(MAX_NODES);
static_assert(pairs(0) == 0 && pairs(1) == 4 && pairs(4) == 16 && pairs(5) == 24 && pairs(64) == 2176, "row starts");

// The walk to the root and what follows it take eight lanes a node, four nodes a warp; all lanes of a warp make
// the calls, with node >= n for none.

// The token rows b and q of a lane: channels 4 (sub + 8 j) + c, sub = lane & 7.
template <typename Tok, int K>
struct Rows {
    Raw<Tok, 4> b[K / 32], q[K / 32];
    __device__ __forceinline__ void load(const Tok *pb, const Tok *pq, int lo, int H, int head, int node, int n, int lane) {
        const size_t row = ((size_t)(lo + (node < n ? node : 0)) * H + head) * K + 4 * (lane & 7);
#pragma unroll
        for (int j = 0; j < K / 32; ++j) b[j].load(pb + row + 32 * j), q[j].load(pq + row + 32 * j);
    }
};

// Sums of eight values over the eight lanes of a node: on return lane `sub` holds the total of x[sub].
__device__ __forceinline__ float node_sums(const float (&x)[8], int lane) {
    float a[4], b[2];
    const bool up4 = lane & 4, up2 = lane & 2, up1 = lane & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a[i] = (up4 ? x[i + 4] : x[i]) + __shfl_xor_sync(0xffffffffu, up4 ? x[i] : x[i + 4], 4);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        b[i] = (up2 ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, up2 ? a[i] : a[i + 2], 2);
    return (up1 ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, up1 ? b[0] : b[1], 1);
}

// From a node to its root, four ancestors at a time.  On return e and g are e_n G_n and q_n G_n at the lane's
// channels, the node's rows of A and P (cA, cP), of anc (whom each is for) and of where (the start of that one's
// row) are written, and the number of ancestors is returned.  sk, sa: k and alpha of all nodes in shared memory.
// Four operations a channel for each pair (node, ancestor), two channels an instruction, the decays multiplied
// in as the walk goes up, and seven shuffles for four pairs.
template <typename Tok, int K, typename SharedTok, typename Parent>
__device__ __forceinline__ int walk(const Rows<Tok, K> &rows, const SharedTok *sk, const float *sa, const Parent *parent,
                                    float *cA, float *cP, unsigned char *anc, unsigned short *where, int node, int n,
                                    int lane, f32x2 (&e)[K / 32][2], f32x2 (&g)[K / 32][2]) {
    constexpr int RJ = K / 32;
    const int sub = lane & 7;
    const auto key = [&](int at, int j, f32x2 (&x)[2]) {
        Raw<SharedTok, 4> r;
        float y[4];
        r.load(sk + at * K + 4 * (sub + 8 * j));
        r.get(y);
        x[0] = pack2(y[0], y[1]);
        x[1] = pack2(y[2], y[3]);
    };
    int at = node < n ? node : -1, above = -1;
#pragma unroll
    for (int j = 0; j < RJ; ++j) {
        f32x2 kk[2];
        float x[4];
        key(at < 0 ? 0 : at, j, kk);
        rows.b[j].get(x);
        e[j][0] = mul2(pack2(x[0], x[1]), kk[0]);
        e[j][1] = mul2(pack2(x[2], x[3]), kk[1]);
        rows.q[j].get(x);
        g[j][0] = pack2(x[0], x[1]);
        g[j][1] = pack2(x[2], x[3]);
    }
    int out = pairs(at < 0 ? 0 : at), root = 0;
    while (__any_sync(0xffffffffu, at >= 0)) {
        float x[8];   // A and P of four pairs
        const bool some = at >= 0;
        int whom = 0;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            x[s] = x[4 + s] = 0.f;
            if (at >= 0) {
                const int up = parent[at];
                f32x2 a[2] = {0ull, 0ull}, p[2] = {0ull, 0ull};
#pragma unroll
                for (int j = 0; j < RJ; ++j) {
                    f32x2 kk[2], aa[2];
                    key(at, j, kk);
                    load2(sa + at * K + 4 * (sub + 8 * j), aa);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        a[c] = fma2(e[j][c], kk[c], a[c]);
                        p[c] = fma2(g[j][c], kk[c], p[c]);
                        e[j][c] = mul2(e[j][c], aa[c]);
                        g[j][c] = mul2(g[j][c], aa[c]);
                    }
                }
                const float2 ya = unpack2(add2(a[0], a[1])), yp = unpack2(add2(p[0], p[1]));
                x[s] = ya.x + ya.y;
                x[4 + s] = yp.x + yp.y;
                root = at;
                at = up;
                ++above;
            }
            if (s == (sub & 3)) whom = root;
        }
        const float sum = node_sums(x, lane);
        if (some) {
            (sub < 4 ? cA : cP)[out + (sub & 3)] = sum;   // the node's own A is not used
            if (sub < 4) {
                anc[out + sub] = (unsigned char)whom;
                where[out + sub] = (unsigned short)pairs(whom);
            }
            out += 4;
        }
    }
    return above;
}

// The deltas eliminated: with p_0 = n, p_1, ... the path from n to its root and R[i] = u_i - S^T (e_i G_i),
//   o_n = S^T (q_n G_n) + sum_j C[n,j] R[p_j],   C[n,j] = P[n,p_j] - sum_{m < j} C[n,m] A[p_m, p_j]
// A node's C needs no other node's, so the columns' work has no order among the nodes left: one product for
// each pair, in place of two and a barrier for each level of the tree.  Lane `sub` takes j = 8 h + sub; the
// coefficients of a finished j go to the others by a shuffle, those of finished blocks of eight through
// shared memory.  All walks of the item must be done; cC may be cP.
__device__ __forceinline__ void eliminate(const float *cA, const float *cP, const unsigned short *where, float *cC,
                                          int node, int n, int above, int lane) {
    const int sub = lane & 7, base = node < n ? pairs(node) : 0;
    if (node >= n) above = -1;
    const int most = __reduce_max_sync(0xffffffffu, above);
    for (int h = 0; h <= most; h += 8) {
        const int j = h + sub;
        const bool mine = j <= above;
        float c = mine ? cP[base + j] : 0.f, up[8];
#pragma unroll
        for (int m = 0; m < 8; ++m) up[m] = mine && m < sub ? cA[where[base + h + m] + sub - m] : 0.f;
        if (mine)
#pragma unroll 4
            for (int m = 0; m < h; ++m) c = fmaf(-cC[base + m], cA[where[base + m] + j - m], c);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            const float done = __shfl_sync(0xffffffffu, c, (lane & 24) | m);
            if (m < sub) c = fmaf(-done, up[m], c);
        }
        if (j <= (above | 3)) cC[base + j] = mine ? c : 0.f;   // with the zeros that fill the row up
        __syncwarp();
    }
}

}  // namespace tree
}  // namespace gdn2
