// Drafted tokens in a tree over a state cache: the read-out of every node, the cache unchanged (sm_100a;
// page "NVIDIA представила Gated DeltaNet-2 ...", section "Техническая схема", the state-update equation, and
// the paragraph on the chunkwise WY form).
//
// A node's state is its parent's after one step of the recurrence; a root's parent is the cached state S.
// With G_n the channel-wise product of the decays on the path from S to n (n's own included), e = b k and
// u = w v, the states need not be formed:
//   delta_n = u_n - S^T (e_n G_n) - sum over proper ancestors i of A[n,i] delta_i,   A[n,i] = sum_c e_n (G_n / G_i) k_i
//   o_n     = S^T (q_n G_n) + sum over ancestors i and n itself of P[n,i] delta_i,   P[n,i] = sum_c q_n (G_n / G_i) k_i
// G_n / G_i is the product of the decays below i down to n.  While every G on n's path is in fp32's range, A and P
// are products of e_n G_n and q_n G_n with k_i / G_i; where one is not (long or hard decays, zero included) the
// decays are multiplied in on the way up instead, without a division.  Which it is goes by the path alone, and
// nothing of another branch is touched.  The deltas are then eliminated (eliminate()), which leaves o_n as a sum
// over n's path alone.
#include "gdn2_tree.cuh"

namespace gdn2 {
namespace tree {

// A lane's channels are 4 (sub + 8 j) + c, sub = lane & 7.

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

// G_n, the product of the decays on a node's path, at the lane's channels.  sa: alpha of all nodes in shared
// memory.
template <int K>
__device__ __forceinline__ void climb(const float *sa, const unsigned char *anc, bool go, int node, int above, int lane,
                                      f32x2 (&G)[K / 32][2]) {
    const int sub = lane & 7, base = pairs(go ? node : 0), most = __reduce_max_sync(0xffffffffu, go ? above : -1);
#pragma unroll
    for (int j = 0; j < K / 32; ++j) G[j][0] = G[j][1] = pack2(1.f, 1.f);
#pragma unroll 1
    for (int h = 0; h <= most; h += 4) {
        if (!go || h > above) continue;
        const uchar4 whom = *reinterpret_cast<const uchar4 *>(anc + base + h);
        const int at[4] = {whom.x, whom.y, whom.z, whom.w};
#pragma unroll
        for (int s = 0; s < 4; ++s)
            if (h + s <= above)
#pragma unroll
                for (int j = 0; j < K / 32; ++j) {
                    f32x2 aa[2];
                    load2(sa + at[s] * K + 4 * (sub + 8 * j), aa);
                    G[j][0] = mul2(G[j][0], aa[0]);
                    G[j][1] = mul2(G[j][1], aa[1]);
                }
    }
}

// A and P of a node's path, to cA and cP, where all its G are in range:  A[n,i] = sum_c (e_n G_n) (k_i / G_i), two
// operations a channel, no chain from one ancestor to the next, and seven shuffles for four pairs.  sk: k_i / G_i of
// all nodes in shared memory; e, g: e_n G_n and q_n G_n.
template <int K>
__device__ __forceinline__ void couple(const float *sk, const unsigned char *anc, float *cA, float *cP, bool go, int node,
                                       int above, int lane, const f32x2 (&e)[K / 32][2], const f32x2 (&g)[K / 32][2]) {
    const int sub = lane & 7, base = pairs(go ? node : 0), most = __reduce_max_sync(0xffffffffu, go ? above : -1);
#pragma unroll 1
    for (int h = 0; h <= most; h += 4) {
        float x[8];
        const bool some = go && h <= above;
        const uchar4 whom = some ? *reinterpret_cast<const uchar4 *>(anc + base + h) : make_uchar4(0, 0, 0, 0);
        const int at[4] = {whom.x, whom.y, whom.z, whom.w};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            f32x2 a[2] = {0ull, 0ull}, p[2] = {0ull, 0ull};
#pragma unroll
            for (int j = 0; j < K / 32; ++j) {
                f32x2 kk[2];
                load2(sk + at[s] * K + 4 * (sub + 8 * j), kk);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    a[c] = fma2(e[j][c], kk[c], a[c]);
                    p[c] = fma2(g[j][c], kk[c], p[c]);
                }
            }
            const float2 ya = unpack2(add2(a[0], a[1])), yp = unpack2(add2(p[0], p[1]));
            x[s] = ya.x + ya.y;
            x[4 + s] = yp.x + yp.y;
        }
        const float sum = node_sums(x, lane);
        if (some) (sub < 4 ? cA : cP)[base + h + (sub & 3)] = sum;   // the node's own A is not used
    }
}

// The kernel on CUDA cores, any type and size.  One block per (column range, head, sequence); the first
// cols / 16 warps own 16 columns of the state each, every warp takes part in the rest.  For a few nodes a chain of
// latencies (8 nodes of one user, H16: 8.1 us with cold caches, 5.8 a call behind another; the columns over 128 SMs),
// for many the 2 n d_k d_v FMA of a head and their shared-memory loads (32 users with 32 nodes: 63 us, against 31 on
// the tensor cores; 128 users of 32 nodes with 128-64 heads 130, of 64 nodes with 64-64 heads 253 and in fp32 547, where
// the FMA alone would take 30, 30 and 121: a block's stages follow one another, and at 64 nodes it has an SM to itself).
template <typename Tok, int K, int V>
__global__ void __launch_bounds__(256, 2) tree_kernel(const Tok *__restrict__ q, const Tok *__restrict__ k,
                                                   const Tok *__restrict__ v, const float *__restrict__ alpha,
                                                   const Tok *__restrict__ b, const Tok *__restrict__ w,
                                                   const float *__restrict__ S, long long slot_stride, int num_slots,
                                                   const int *__restrict__ slots, const int *__restrict__ cu,
                                                   const int *__restrict__ parents, Tok *__restrict__ o, int H,
                                                   int splits, int total, int max_nodes, unsigned *status) {
    constexpr int RJ = K / 32;
    extern __shared__ __align__(16) float smem[];
    behind_last_kernel();
    // splits, cols and groups are powers of two: shifts, where a division by them takes as long as a load
    const int split_bits = __ffs(splits) - 1, cols = V >> split_bits, tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int head = blockIdx.x >> split_bits, col0 = (blockIdx.x & (splits - 1)) * cols, seq = blockIdx.y;
    float *sk = smem, *sa = sk + max_nodes * K, *se = sa + max_nodes * K, *sq = se + max_nodes * K;   // sk: k / G
    float *sr = sq + max_nodes * K, *ss = sr + max_nodes * cols;
    float *cA = ss + max_nodes * cols, *cP = cA + pairs(max_nodes);
    int *sp = reinterpret_cast<int *>(cP + pairs(max_nodes));
    unsigned char *anc = reinterpret_cast<unsigned char *>(sp + max_nodes), *depth = anc + pairs(max_nodes),
                  *fine = depth + max_nodes;

    const int lo = cu[seq], hi = cu[seq + 1], slot = slots[seq];
    unsigned bad = 0;
    if (lo < 0 || hi < lo || hi > total || hi - lo > max_nodes) bad = DEV_RANGE;
    else if (slot < -1 || slot >= num_slots) bad = DEV_SLOT;

    // Everything is on its way before the first barrier: the state to registers, the tokens as they are stored to where
    // their products with the decays will stand.
    // The warp's slice of the state: rows 4 (rg + 8 j) + i, columns c0 .. c0 + 3; where there are more warps than
    // column groups they share the nodes.
    const int groups = cols / 16, group_bits = __ffs(groups) - 1, shares = nt >> 5 >> group_bits;
    const int rg = lane >> 2, c0 = (warp & (groups - 1)) * 16 + (lane & 3) * 4;
    float s[RJ][4][4];
#pragma unroll
    for (int j = 0; j < RJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (slot >= 0 && !bad)
                x = ld_stream(reinterpret_cast<const float4 *>(S + (size_t)slot * slot_stride + (size_t)head * K * V +
                                                               (size_t)(4 * (rg + 8 * j) + i) * V + col0 + c0));
            s[j][i][0] = x.x; s[j][i][1] = x.y; s[j][i][2] = x.z; s[j][i][3] = x.w;
        }
    const int n = bad ? 0 : hi - lo;
    if (tid < n) {
        const int p = parents[lo + tid];
        if (p < -1 || p >= tid) bad = DEV_PARENT;
        sp[tid] = p;
    }
    constexpr int TOK = sizeof(Tok);
    Tok *raw_v = reinterpret_cast<Tok *>(TOK == 4 ? sr : ss), *raw_w = reinterpret_cast<Tok *>(ss) + (TOK == 4 ? 0 : cols);
    const int pitch = cols * 4 / TOK;   // of a node's v and w: bf16 ones share a row of ss
    for (int node = warp; node < n; node += nt >> 5) {   // a warp a node, 16 bytes a lane
        const size_t row = (size_t)(lo + node) * H + head;
        const auto bring = [&](void *to, const void *from, int at) {
            cp_async16((uint32_t)__cvta_generic_to_shared(to) + at, static_cast<const char *>(from) + at);
        };
        constexpr int CHUNKS = TOK * K / 16;   // of a row of k, b or q
#pragma unroll
        for (int i = 0; i < K / 4; i += 32)
            if (i + lane < K / 4) bring(sa + node * K, alpha + row * K, 16 * (i + lane));
#pragma unroll
        for (int i = 0; i < 3 * CHUNKS; i += 32) {
            const int which = (i + lane) / CHUNKS, at = 16 * ((i + lane) % CHUNKS);
            if (which < 3) bring((which == 0 ? sk : which == 1 ? se : sq) + node * K, (which == 0 ? k : which == 1 ? b : q) + row * K, at);
        }
        const int chunks = TOK * cols / 16;
        for (int i = lane; i < 2 * chunks; i += 32)
            if (i < chunks) bring(raw_v + node * pitch, v + row * V + col0, 16 * i);
            else bring(raw_w + node * pitch, w + row * V + col0, 16 * (i - chunks));
    }
    cp_async_wait();
    if (__syncthreads_or(bad != 0)) {
        if (bad) atomicOr(status, bad);
        return;
    }
    if (n == 0) return;
    for (int i = tid; i < n * (cols / 4); i += nt) {   // u, until the product is taken off it
        const int at = (i >> (group_bits + 2)) * pitch + (i & (cols / 4 - 1)) * 4;
        Raw<Tok, 4> rv, rw;
        float x[4], y[4];
        rv.load(raw_v + at);
        rw.load(raw_w + at);
        rv.get(x);
        rw.get(y);
        *reinterpret_cast<float4 *>(sr + 4 * i) = make_float4(x[0] * y[0], x[1] * y[1], x[2] * y[2], x[3] * y[3]);
    }
    if (tid < n) depth[tid] = (unsigned char)list_path(sp, anc, tid);
    __syncthreads();
    for (int n0 = warp * 4; n0 < n; n0 += nt / 8) {
        const int node = n0 + (lane >> 3), sub = lane & 7;
        Raw<Tok, 4> rk[RJ], rb[RJ], rq[RJ];
        if (node < n)
#pragma unroll
            for (int j = 0; j < RJ; ++j) {
                rk[j].load(reinterpret_cast<const Tok *>(sk + node * K) + 4 * (sub + 8 * j));
                rb[j].load(reinterpret_cast<const Tok *>(se + node * K) + 4 * (sub + 8 * j));
                rq[j].load(reinterpret_cast<const Tok *>(sq + node * K) + 4 * (sub + 8 * j));
            }
        __syncwarp();   // before the first of the node's lanes writes over them
        f32x2 G[RJ][2];
        climb<K>(sa, anc, node < n, node, node < n ? depth[node] : -1, lane, G);
        const bool good = in_range<K>(G, lane);
        if (node < n) {
            if (sub == 0) fine[node] = good;
#pragma unroll
            for (int j = 0; j < RJ; ++j) {
                const int at = node * K + 4 * (sub + 8 * j);
                const float2 g0 = unpack2(G[j][0]), g1 = unpack2(G[j][1]);
                float kk[4], bb[4], qq[4];
                rk[j].get(kk);
                rb[j].get(bb);
                rq[j].get(qq);
                *reinterpret_cast<float4 *>(se + at) = make_float4(bb[0] * kk[0] * g0.x, bb[1] * kk[1] * g0.y,
                                                                   bb[2] * kk[2] * g1.x, bb[3] * kk[3] * g1.y);
                *reinterpret_cast<float4 *>(sq + at) = make_float4(qq[0] * g0.x, qq[1] * g0.y, qq[2] * g1.x, qq[3] * g1.y);
                // used where G is in range only: two units in the last place there, as the products' own roundings together
                *reinterpret_cast<float4 *>(sk + at) =
                    make_float4(__fdividef(kk[0], g0.x), __fdividef(kk[1], g0.y), __fdividef(kk[2], g1.x), __fdividef(kk[3], g1.y));
            }
        }
    }
    __syncthreads();
    for (int n0 = warp * 4; n0 < n; n0 += nt / 8) {
        const int node = n0 + (lane >> 3), sub = lane & 7, above = node < n ? depth[node] : -1;
        bool good = true;
        for (int j = sub; j <= above; j += 8) good = good && fine[anc[pairs(node) + j]];
        good = (__ballot_sync(0xffffffffu, good) >> (lane & 24) & 0xffu) == 0xffu;
        f32x2 e[RJ][2], g[RJ][2];
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
            load2(se + (node < n ? node : 0) * K + 4 * (sub + 8 * j), e[j]);
            load2(sq + (node < n ? node : 0) * K + 4 * (sub + 8 * j), g[j]);
        }
        couple<K>(sk, anc, cA, cP, node < n && good, node, above, lane, e, g);
        if (__any_sync(0xffffffffu, node < n && !good))
            couple_far<Tok, K>(q, k, b, alpha, anc, cA, cP, node < n && !good, lo, H, head, node, above, lane);
    }
    __syncthreads();
    for (int n0 = warp * 4; n0 < n; n0 += nt / 8) {
        const int node = n0 + (lane >> 3);
        eliminate(cA, cP, anc, cP, node < n, node, node < n ? depth[node] : 0, lane);
    }

    // S^T (e G) and S^T (q G) of every node
#pragma unroll 2
    for (int t = warp >> group_bits; t < n; t += shares) {
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
        const float sum = scatter_sum8(p, lane);   // of p[rg]
        const int at = t * cols + c0 + (rg & 3);
        if (rg < 4) sr[at] -= sum;
        else ss[at] = sum;
    }
    __syncthreads();

    // o: four columns a thread, the nodes in turn over the block
    const size_t first = ((size_t)lo * H + head) * V + col0;
    for (int i = tid; i < n * (cols / 4); i += nt) {
        const int node = i >> (group_bits + 2), col = (i & (cols / 4 - 1)) * 4, base = pairs(node), above = depth[node];
        float4 x = *reinterpret_cast<const float4 *>(ss + 4 * i);
#pragma unroll 4
        for (int j = 0; j <= above; ++j) {
            const float c = cP[base + j];
            const float4 r = *reinterpret_cast<const float4 *>(sr + anc[base + j] * cols + col);
            x.x = fmaf(c, r.x, x.x); x.y = fmaf(c, r.y, x.y); x.z = fmaf(c, r.z, x.z); x.w = fmaf(c, r.w, x.w);
        }
        Tok *out = o + first + (size_t)node * H * V + col;
        store_tok(out, x.x); store_tok(out + 1, x.y); store_tok(out + 2, x.z); store_tok(out + 3, x.w);
    }
}

template <typename Tok, int K, int V>
int launch_t(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
             const float *S, long long slot_stride, int num_slots, const int *slots, const int *cu, const int *parents,
             void *o, int batch, int H, int total, int max_nodes, unsigned *status, cudaStream_t st) {
    const auto smem = [&](int n, int cols) {
        return sizeof(float) * (size_t)n * (4 * K + 2 * cols) + (2 * sizeof(float) + 1) * (size_t)pairs(n) +
               (sizeof(int) + 2) * (size_t)n;
    };
    // few chains: their columns over more SMs
    int splits = 1;
    while (splits < V / 16 && (long long)batch * H * splits * 2 <= 148) splits *= 2;
    const int cols = V / splits;
    // Two threads a column at least; eight warps for the nodes where there is no third block an SM that they would keep
    // out, for want of blocks or of shared memory (us, 128 threads / 256; H x nodes, d_k-d_v: 1 user 16 x 24, 128-128
    // bf16 10.7 / 8.2; 2 users 8 x 64, 128-128 fp32 26.9 / 17.9; 128 users 16 x 32, 128-64 bf16 166 / 135; where there is
    // one, 128 users 16 x 12, 64-64 bf16 35.8 / 46.2).
    const long long blocks = (long long)H * splits * batch;
    const int threads = max_nodes > 8 && (blocks <= 2 * 148 || 3 * smem(max_nodes, cols) > 227 * 1024) ? 256
                        : 2 * cols < 128                                                             ? 128
                                                                                                     : 2 * cols;
    if (!allow_smem(tree_kernel<Tok, K, V>, smem(MAX_NODES, V))) return -6;
    return launch_close(tree_kernel<Tok, K, V>, dim3(H * splits, batch), threads, smem(max_nodes, cols),
                        st, (const Tok *)q, (const Tok *)k, (const Tok *)v, alpha, (const Tok *)b, (const Tok *)w, S, slot_stride,
                        num_slots, slots, cu, parents, (Tok *)o, H, splits, total, max_nodes, status);
}

// Which kernel: the tensor-core one's period for an item hardly depends on its nodes (5.2 us an SM for four, 10.3 for 64),
// this one's grows with them, and few items have their columns over all SMs here.  H16, us, this / that, one call behind
// another; [with cold caches, device time]:
//   1 user     24 nodes  7.8 /  9.1 [10.3 / 13.1]   32 nodes  9.7 /  9.9                   40 nodes  14.1 / 12.0 [16.7 / 16.3]
//   2 users    20 nodes  8.3 /  9.0                 24 nodes  8.7 /  9.1 [11.3 / 13.5]   32 nodes  10.8 / 10.0
//   4 users    12 nodes  8.0 /  8.3                 16 nodes  8.8 /  8.5 [11.7 / 12.8]   20 nodes  10.1 /  9.1
//   8 users     8 nodes  8.4 /  8.3 [10.9 / 12.1]   10 nodes  9.2 /  8.8                   16 nodes  11.6 /  8.7 [14.8 / 13.2]
//   32 users    7 nodes 19.6 / 20.2                  8 nodes 20.6 / 20.1 [24.8 / 25.0]   10 nodes  23.8 / 20.6
//   128 users   6 nodes 64.9 / 69.4                  7 nodes 68.7 / 69.8                    8 nodes  73.0 / 70.2 [77.3 / 74.1]
//   with cold caches alone: 32 users of 32 nodes [62.9 / 31.2], 128 of 16 [116.5 / 76.5], of 64 [535.5 / 142.8]
bool use_tc(int batch, int H, int max_nodes) {
    const long long items = (long long)batch * H;
    return max_nodes > (items > 148 ? 7 : items > 64 ? 9 : items > 32 ? 15 : items > 16 ? 20 : 40);
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
    if (bf16 && K == 128 && V == 128 && tree::use_tc(batch, H, max_nodes)) return go(tree::launch_tc);
    if (bf16) {
        if (K == 128) return V == 128 ? go(tree::launch_t<__nv_bfloat16, 128, 128>) : go(tree::launch_t<__nv_bfloat16, 128, 64>);
        return V == 128 ? go(tree::launch_t<__nv_bfloat16, 64, 128>) : go(tree::launch_t<__nv_bfloat16, 64, 64>);
    }
    if (K == 128) return V == 128 ? go(tree::launch_t<float, 128, 128>) : go(tree::launch_t<float, 128, 64>);
    return V == 128 ? go(tree::launch_t<float, 64, 128>) : go(tree::launch_t<float, 64, 64>);
}

}  // namespace gdn2
