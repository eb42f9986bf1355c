// Drafted trees over a state cache on the tensor cores (sm_100a): bf16 tokens, d_k = d_v = 128.  The formulas are
// those of gdn2_tree.cu; what is different is where the two products with the state run, and that a
// persistent CTA's warps work on several (sequence, head) items at once.
//
// S^T [e G; q G]^T, 128 x 128 x 2n, is 2 n 128^2 FMA a head, more than CUDA cores do in the time that HBM takes
// for the state and the tokens from five nodes on.  Both factors are split into two bf16, x = hi + lo (16
// significant bits, relative error 2^-17): three tcgen05 products hi hi + hi lo + lo hi keep the error far
// below the rounding of the bf16 output, where one product of bf16 operands would double that rounding.  Of trees of 64
// nodes o is 2e-6 of its norm off before that rounding (1.66e-3; the fp32 kernel: 1e-7), nearly all of it by the couplings
// and 4e-7 by the products with the state; against fp64 its error is 1.658277e-3 where plain fp32's is 1.658276e-3.
// (4e-6 while P of a node with itself, which has no decay in it, was a product of those two as well, in place of q k in
// fp32: 134 us for the full batch, 136 now.  The parent's couplings in fp32 too would leave 6e-7, for 145 to 148 us.  Slow
// decays keep 4e-6, distant couplings then counting like near ones.  The lo lo products would take a fifth off.  Three bf16
// would end it, but their images, 48 KB more, do not fit beside the others; couplings on CUDA cores take a third more time.)
//   state group  (4 warps)  a column of S a thread, split, into tensor memory: the A operand S^T, lane = value
//                           column, two buffers
//   path group   (8 warps)  G, a channel a thread from parents to children; then, eight lanes a node, the rows
//                           e G, q G and k / G, split, into swizzled images
//   pair group   (8 warps)  [e G; q G] [k / G]^T, 2n x 128 x n and split alike, holds A and P of all pairs of nodes:
//                           from tensor memory (lane = row) those of the paths to lists, then the elimination
//   column group (8 warps)  R = u - S^T (e G) and S^T (q G) from tensor memory (lane = value column) to shared
//                           memory, then o = S^T (q G) + C R, two nodes a warp and eight columns a lane
//   scout warp              reads and checks the items, lists their paths, brings the tokens' lines into L2 ahead
//                           of the groups
//   lead warp               issues the products
// 128 trees of 64 nodes, H16, take 137 us for 403 MB (device time, cold caches; 136 one call behind another): 9.9 us an
// item, of which memory needs 4.5.  Half of the issue slots are taken, by the splitting of the operands, the decays, the
// elimination and the sums; with the pairs on CUDA cores in one group with the paths it took 191 us, with those in groups
// of their own 181, when this took 146.  960 threads leave 64 registers each, and the path and pair groups spill (44 bytes
// of stores, 72 of loads a thread).  Few items (32 trees of up to 32 nodes: 29 us, 25 one call behind another) wait for
// the chain of one.
#include "gdn2_tree.cuh"
#include "tc_ptx.cuh"

namespace gdn2 {
namespace tree {

using namespace gdn2::tc;

constexpr int D = 128;
constexpr int COLUMN_WARPS = 8, STATE_WARPS = 4, PATH_WARPS = 8, PAIR_WARPS = 8;   // in this order; then the lead and the scout
constexpr int PATH0 = COLUMN_WARPS + STATE_WARPS, PAIR0 = PATH0 + PATH_WARPS, LEAD = PAIR0 + PAIR_WARPS,
              SCOUT = LEAD + 1, TC_THREADS = 32 * (SCOUT + 1);
constexpr int METAS = 3;
constexpr uint32_t BAR_COLUMN = 1, BAR_PATH = 2, BAR_PAIR = 3, BAR_STATE = 4, WAIT_LIMIT = 1u << 20;
constexpr uint32_t TM_S = 0, TM_D = 256, TM_P = 384, TM_COLS = 512;   // S: two buffers of hi (64 columns) and lo (64)

// An item: its nodes lo .. lo+n-1, the state's slot, the nodes' parents, paths and numbers of ancestors, and the
// nodes by that number, the deepest first (so that the nodes of a warp take about as many steps).
struct Meta {
    int lo, n, slot, head;
    signed char parent[MAX_NODES];
    unsigned char anc[MAX_PAIRS], above[MAX_NODES], order[MAX_NODES];
    unsigned char fine[MAX_NODES];   // whether a node's G is in range (the path group's)
};

struct TcShared {
    unsigned char b_hi[2 * MAX_NODES * D * 2], b_lo[2 * MAX_NODES * D * 2];   // [e G; q G], swizzled
    unsigned char k_hi[MAX_NODES * D * 2], k_lo[MAX_NODES * D * 2];           // k / G
    float alpha[MAX_NODES][D];                // then G
    float r[MAX_NODES][D], x[MAX_NODES][D];   // u, then R; S^T (q G); by node and value column
    float a[MAX_PAIRS], c[2][MAX_PAIRS];      // A; P, then C
    Meta meta[METAS];
    float own[2][MAX_NODES];                  // P of a node with itself, q k
    unsigned long long path[MAX_NODES];       // a bit for each node on a node's path
    unsigned long long meta_known[METAS], meta_full[METAS], meta_free[METAS], s_full[2], s_free[2], coef_full[2], coef_free[2], b_full, b_free,
        d_full, d_free, p_full, p_free;
    uint32_t tmem, abort;
};
static_assert(sizeof(TcShared) + 1024 <= 227 * 1024, "shared memory of an SM");

// x = hi + lo, two values at a time as packed bf16 (the first in the low half).  An infinity leaves a NaN in lo:
// what it meets is not finite either way.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(x, y);
    lo = pack_bf16(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}

// Which of the nodes, the deepest first, eight lanes take in a round: the shallowest behind the deepest.
__device__ __forceinline__ int place_of(int round, int team) { return round ? MAX_NODES - 1 - team : team; }

__device__ __forceinline__ float inverse(float x) {   // to one unit of fp32
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__global__ void __launch_bounds__(TC_THREADS, 1) tree_tc_kernel(
    const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ k, const __nv_bfloat16 *__restrict__ v,
    const float *__restrict__ alpha, const __nv_bfloat16 *__restrict__ b, const __nv_bfloat16 *__restrict__ w,
    const float *__restrict__ S, long long slot_stride, int num_slots, const int *__restrict__ slots,
    const int *__restrict__ cu, const int *__restrict__ parents, __nv_bfloat16 *__restrict__ o, int batch, int H,
    int total, int max_nodes, uint32_t limit, unsigned *status) {
    extern __shared__ unsigned char raw[];
    TcShared &sh = *reinterpret_cast<TcShared *>(raw + ((1024 - (smem_u32(raw) & 1023)) & 1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long items = (long long)batch * H;
    const auto bar = [](unsigned long long &x) { return smem_u32(&x); };
    volatile uint32_t *abort = &sh.abort;

    if (tid == 0) {
        for (int i = 0; i < METAS; ++i) mbar_init(bar(sh.meta_known[i]), 1), mbar_init(bar(sh.meta_full[i]), 1), mbar_init(bar(sh.meta_free[i]), SCOUT);   // a warp each, but the scout
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(sh.s_full[i]), STATE_WARPS);
            mbar_init(bar(sh.s_free[i]), 1);
            mbar_init(bar(sh.coef_full[i]), PAIR_WARPS);
            mbar_init(bar(sh.coef_free[i]), COLUMN_WARPS);
        }
        mbar_init(bar(sh.b_full), PATH_WARPS);
        mbar_init(bar(sh.b_free), 1);
        mbar_init(bar(sh.d_full), 1);
        mbar_init(bar(sh.d_free), COLUMN_WARPS);
        mbar_init(bar(sh.p_full), 2);   // the products, and the lead for what the path group wrote
        mbar_init(bar(sh.p_free), PAIR_WARPS);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    behind_last_kernel();   // and only then tensor memory, which it may hold
    if (warp == LEAD) tmem_alloc(smem_u32(&sh.tmem), TM_COLS);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem;

    // Every wait is bounded, and every thread of a group gets the same verdict, so that none is left at one of
    // the group's barriers.  One warp of a group polls, the others sleep at the barrier.  Phases count the items
    // that have nodes (c); the others only pass their meta on.
    const auto wait = [&](unsigned long long &x, int phase) {
        const bool ok = mbar_wait(bar(x), phase & 1, limit) && !*abort;
        if (!ok) *abort = 1u;
        return ok;
    };
    const int poller = warp < COLUMN_WARPS ? 0 : warp < PATH0 ? COLUMN_WARPS : warp < PAIR0 ? PATH0 : PAIR0;
    const auto group_wait = [&](unsigned long long &x, int phase, uint32_t id, uint32_t threads) {
        const bool ok = !group_or(id, threads, warp == poller && !wait(x, phase));
        fence_after();
        return ok;
    };
    const auto warp_wait = [&](unsigned long long &x, int phase) { return !__any_sync(0xffffffffu, !wait(x, phase)); };
    const auto arrive = [&](unsigned long long &x) {   // once for the warp
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(x));
    };

    int c = 0;
    if (warp == SCOUT) {
        // an item a turn: its sequence and head without a division
        int seq = blockIdx.x / (unsigned)H, head = blockIdx.x % (unsigned)H;
        const int seqs_on = gridDim.x / (unsigned)H, heads_on = gridDim.x % (unsigned)H;
        for (int it = 0;; ++it) {
            if (blockIdx.x + (long long)it * gridDim.x >= items || !warp_wait(sh.meta_free[it % METAS], it / METAS + 1)) break;
            Meta &m = sh.meta[it % METAS];
            const int lo = cu[seq], hi = cu[seq + 1], slot = slots[seq];
            unsigned bad = 0;
            if (lo < 0 || hi < lo || hi > total || hi - lo > max_nodes) bad = DEV_RANGE;
            else if (slot < -1 || slot >= num_slots) bad = DEV_SLOT;
            int n = bad ? 0 : hi - lo;
            for (int i = lane; i < n; i += 32) {
                const int p = parents[lo + i];
                if (p < -1 || p >= i) bad |= DEV_PARENT;
                else m.parent[i] = (signed char)p;
            }
            bad = __reduce_or_sync(0xffffffffu, bad);
            if (bad) {
                if (lane == 0) atomicOr(status, bad);
                n = 0;
            }
            if (lane == 0) m.lo = lo, m.n = n, m.slot = slot, m.head = head;
            arrive(sh.meta_known[it % METAS]);   // all but the pair group go on with that
            // a line a lane (bulk prefetches of whole rows took 60 cycles each, 24,000 for 64 nodes)
            for (int i = lane; i < 2 * n; i += 32) {
                const size_t row = ((size_t)(lo + i / 2) * H + head) * D + i % 2 * 64;
                prefetch_l2(k + row);
                prefetch_l2(b + row);
                prefetch_l2(q + row);
                prefetch_l2(v + row);
                prefetch_l2(w + row);
                prefetch_l2(alpha + row);
                prefetch_l2(alpha + row + 32);
            }
            int above[2] = {-1, -1};
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (lane + 32 * r < n) m.above[lane + 32 * r] = (unsigned char)(above[r] = list_path(m.parent, m.anc, lane + 32 * r));
            int place = 0;
            for (int l = __reduce_max_sync(0xffffffffu, max(above[0], above[1])); l >= 0; --l)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const unsigned here = __ballot_sync(0xffffffffu, above[r] == l);
                    if (above[r] == l) m.order[place + __popc(here & ((1u << lane) - 1))] = (unsigned char)(lane + 32 * r);
                    place += __popc(here);
                }
            arrive(sh.meta_full[it % METAS]);
            seq += seqs_on;
            head += heads_on;
            if (head >= H) head -= H, ++seq;
        }
    } else if (warp == LEAD) {
        int pairs_out = 0, state_out = 0;   // items whose products have been issued
        for (int it = 0;; ++it) {
            if (blockIdx.x + (long long)it * gridDim.x >= items) break;
            if (!warp_wait(sh.meta_known[it % METAS], it / METAS)) break;
            const int n = sh.meta[it % METAS].n;
            arrive(sh.meta_free[it % METAS]);
            if (n > 0) {
                const int rows = (n + 7) / 8 * 8, cols = (n + 15) / 16 * 16;
                const uint64_t hi = desc_kmajor(smem_u32(sh.b_hi), 2 * MAX_NODES, 0), lo = desc_kmajor(smem_u32(sh.b_lo), 2 * MAX_NODES, 0),
                               k_hi = desc_kmajor(smem_u32(sh.k_hi), MAX_NODES, 0), k_lo = desc_kmajor(smem_u32(sh.k_lo), MAX_NODES, 0);
                // eight steps of 16 channels; the address field counts 16 bytes: 32 bytes a step, and the half's image
                const auto step = [](int rows, int j) { return (j >> 2) * (rows * 128 >> 4) + (j & 3) * 2; };
                if (!warp_wait(sh.b_full, c) || !warp_wait(sh.p_free, c + 1)) break;
                fence_after();
                if (lane == 0) {   // the pairs; what lies behind the rows and columns of nodes is not read
                    const uint32_t idesc = idesc_bf16(128, cols, 0, 0);
                    const auto products = [&](uint64_t a, uint64_t desc, uint32_t acc) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            mma_ss(tmem + TM_P, a + step(2 * MAX_NODES, j), desc + step(MAX_NODES, j), idesc, acc | (j > 0));
                    };
                    products(hi, k_hi, 0);
                    products(lo, k_hi, 1);
                    products(hi, k_lo, 1);
                    mma_commit(bar(sh.p_full));
                    mbar_arrive(bar(sh.p_full));
                }
                ++pairs_out;
                __syncwarp();
                if (!warp_wait(sh.s_full[c & 1], c >> 1) || !warp_wait(sh.d_free, c + 1)) break;
                fence_after();
                if (lane == 0) {
                    const uint32_t idesc = idesc_bf16(128, 2 * rows, 0, 0), s = tmem + TM_S + (c & 1) * 128;
                    const auto products = [&](uint32_t a, uint64_t desc, uint32_t acc) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            mma_ts(tmem + TM_D, a + 8 * j, desc + step(2 * MAX_NODES, j), idesc, acc | (j > 0));
                    };
                    products(s, hi, 0);
                    products(s, lo, 1);
                    products(s + 64, hi, 1);
                    mma_commit(bar(sh.s_free[c & 1]));
                    mma_commit(bar(sh.b_free));
                    mma_commit(bar(sh.d_full));
                }
                ++state_out;
                __syncwarp();
                ++c;
            }
        }
        // The block gives up neither its shared nor its tensor memory before the last products have ended, whatever the
        // other warps' waits came to.
        if (pairs_out && !mbar_wait(bar(sh.p_full), (pairs_out - 1) & 1, WAIT_LIMIT)) *abort = 1u;
        if (state_out && !mbar_wait(bar(sh.d_full), (state_out - 1) & 1, WAIT_LIMIT)) *abort = 1u;
    } else if (warp < COLUMN_WARPS) {
        const int col = tid & 127, half = tid >> 7;   // value column, warpgroup
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        for (int it = 0;; ++it) {
            if (blockIdx.x + (long long)it * gridDim.x >= items) break;
            if (!group_wait(sh.meta_known[it % METAS], it / METAS, BAR_COLUMN, 32 * COLUMN_WARPS)) break;
            const Meta &m = sh.meta[it % METAS];
            const int n = m.n;
            if (n > 0) {
                const size_t first = ((size_t)m.lo * H + m.head) * D;
                // u, eight columns a thread at a time (group_wait's barrier is behind the last item's reads)
#pragma unroll 4
                for (int i = tid; i < n * (D / 8); i += 32 * COLUMN_WARPS) {
                    const size_t at = first + (size_t)(i / (D / 8)) * H * D + i % (D / 8) * 8;
                    Raw<__nv_bfloat16, 8> rv, rw;
                    float x[8], y[8];
                    rv.load(v + at);
                    rw.load(w + at);
                    rv.get(x);
                    rw.get(y);
                    float *to = &sh.r[0][0] + 8 * i;
                    *reinterpret_cast<float4 *>(to) = make_float4(x[0] * y[0], x[1] * y[1], x[2] * y[2], x[3] * y[3]);
                    *reinterpret_cast<float4 *>(to + 4) = make_float4(x[4] * y[4], x[5] * y[5], x[6] * y[6], x[7] * y[7]);
                }
                if (!group_wait(sh.d_full, c, BAR_COLUMN, 32 * COLUMN_WARPS)) break;
                const int rows = (n + 7) / 8 * 8;
                for (int i0 = 0; i0 < n; i0 += 32) {   // one warpgroup each of the two products
                    uint32_t y[32];
                    tmem_ld32(tmem + lanes + TM_D + half * rows + i0, y);
                    wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) {   // the rows behind the last node are not read
                        if (half) sh.x[i0 + i][col] = __uint_as_float(y[i]);
                        else sh.r[i0 + i][col] -= __uint_as_float(y[i]);
                    }
                }
                fence_before();
                arrive(sh.d_free);
                if (!group_wait(sh.coef_full[c & 1], c >> 1, BAR_COLUMN, 32 * COLUMN_WARPS)) break;
                // half a warp takes a node: eight columns a lane, 4 l and 64 + 4 l and the three after each
                for (int i = 2 * warp; i < n; i += 2 * COLUMN_WARPS) {
                    const bool real = i + (lane >> 4) < n;
                    const int node = m.order[real ? i + (lane >> 4) : i], base = pairs(node), above = m.above[node];
                    const int at = 4 * (lane & 15), most = __reduce_max_sync(0xffffffffu, above);
                    f32x2 x[4];
                    load2(&sh.x[node][at], reinterpret_cast<f32x2 (&)[2]>(x[0]));
                    load2(&sh.x[node][64 + at], reinterpret_cast<f32x2 (&)[2]>(x[2]));
                    for (int j = 0; j <= most; j += 4) {
                        if (j > above) continue;
                        const float4 c4 = *reinterpret_cast<const float4 *>(&sh.c[c & 1][base + j]);
                        const uchar4 a4 = *reinterpret_cast<const uchar4 *>(m.anc + base + j);
                        const float cc[4] = {c4.x, c4.y, c4.z, c4.w};
                        const int from[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            f32x2 y[2], z[2];
                            const f32x2 c2 = pack2(cc[s], cc[s]);
                            load2(&sh.r[from[s]][at], y);
                            load2(&sh.r[from[s]][64 + at], z);
                            x[0] = fma2(c2, y[0], x[0]);
                            x[1] = fma2(c2, y[1], x[1]);
                            x[2] = fma2(c2, z[0], x[2]);
                            x[3] = fma2(c2, z[1], x[3]);
                        }
                    }
                    if (real) {
                        __nv_bfloat16 *out = o + first + (size_t)node * H * D + at;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float2 x0 = unpack2(x[2 * h]), x1 = unpack2(x[2 * h + 1]);
                            *reinterpret_cast<uint2 *>(out + 64 * h) = make_uint2(pack_bf16(x0.x, x0.y), pack_bf16(x1.x, x1.y));
                        }
                    }
                }
                arrive(sh.coef_free[c & 1]);
                ++c;
            }
            arrive(sh.meta_free[it % METAS]);
        }
    } else if (warp < PATH0) {
        const int col = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        for (int it = 0;; ++it) {
            if (blockIdx.x + (long long)it * gridDim.x >= items) break;
            if (!group_wait(sh.meta_known[it % METAS], it / METAS, BAR_STATE, 32 * STATE_WARPS)) break;
            const Meta &m = sh.meta[it % METAS];
            const int n = m.n, slot = m.slot, head = m.head;
            arrive(sh.meta_free[it % METAS]);
            if (n == 0) continue;
            const float *src = S + (size_t)(slot < 0 ? 0 : slot) * slot_stride + (size_t)head * D * D + col;
            const uint32_t to = tmem + lanes + TM_S + (c & 1) * 128;
            bool ok = true;
#pragma unroll 1
            for (int part = 0; part < 4; ++part) {
                float x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = slot < 0 ? 0.f : __ldcs(src + (size_t)(32 * part + i) * D);
                if (part == 0 && !(ok = group_wait(sh.s_free[c & 1], (c >> 1) + 1, BAR_STATE, 32 * STATE_WARPS))) break;
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) split2(x[2 * i], x[2 * i + 1], hi[i], lo[i]);
                tmem_st16(to + 16 * part, hi);
                tmem_st16(to + 64 + 16 * part, lo);
            }
            if (!ok) break;
            wait_st();
            fence_before();
            arrive(sh.s_full[c & 1]);
            ++c;
        }
    } else if (warp < PAIR0) {
        constexpr int THREADS = 32 * PATH_WARPS;
        const int t = tid - 32 * PATH0, sub = lane & 7;
        for (int it = 0;; ++it) {
            if (blockIdx.x + (long long)it * gridDim.x >= items) break;
            if (!group_wait(sh.meta_known[it % METAS], it / METAS, BAR_PATH, THREADS)) break;   // and the last item's rows
            Meta &m = sh.meta[it % METAS];
            const int n = m.n, rows = (n + 7) / 8 * 8;
            if (n > 0) {
                const size_t first = ((size_t)m.lo * H + m.head) * D;
                for (int i = t; i < n * (D / 4); i += THREADS)
                    cp_async16(smem_u32(&sh.alpha[0][0]) + 16 * i, alpha + first + (size_t)(i / (D / 4)) * H * D + i % (D / 4) * 4);
                cp_async_wait();
                group_sync(BAR_PATH, THREADS);
                if (t < D) {   // G from parents to children, who stand behind them: four nodes a load latency
                    float *at = &sh.alpha[0][t];
                    float next[4];
                    char4 next4 = *reinterpret_cast<const char4 *>(m.parent);
#pragma unroll
                    for (int i = 0; i < 4; ++i) next[i] = at[i * D];
#pragma unroll 1
                    for (int i0 = 0; i0 < n; i0 += 4) {
                        const int up[4] = {next4.x, next4.y, next4.z, next4.w};
                        float x[4], g[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) g[i] = at[min(max(up[i], 0), i0) * D], x[i] = next[i];
                        const int ahead = min(i0 + 4, MAX_NODES - 4);
                        next4 = *reinterpret_cast<const char4 *>(m.parent + ahead);
#pragma unroll
                        for (int i = 0; i < 4; ++i) next[i] = at[(ahead + i) * D];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
#pragma unroll
                            for (int f = 0; f < i; ++f) g[i] = up[i] == i0 + f ? x[f] : g[i];
                            x[i] *= up[i] < 0 ? 1.f : g[i];
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) at[(i0 + i) * D] = x[i];   // behind the last node: anything
                    }
                }
                if (!group_wait(sh.b_free, c + 1, BAR_PATH, THREADS)) break;   // the products of the item before
#pragma unroll 1
                for (int round = 0; round < 2 && 32 * round < n; ++round) {
                    const int node = 32 * round + (t >> 3);
                    const bool go = node < n;
                    Raw<__nv_bfloat16, 8> rk[2], rb[2], rq[2];
                    const size_t row = first + (size_t)node * H * D + 8 * sub;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        rk[j].clear();
                        rb[j].clear();
                        rq[j].clear();
                        if (go) rk[j].load(k + row + 64 * j), rb[j].load(b + row + 64 * j), rq[j].load(q + row + 64 * j);
                    }
                    f32x2 G[4][2];
#pragma unroll
                    for (int j = 0; j < 4; ++j) load2(&sh.alpha[node][8 * sub + 64 * (j >> 1) + 4 * (j & 1)], G[j]);
                    const bool good = in_range<D>(G, lane);
                    if (!go) continue;
                    if (sub == 0) m.fine[node] = good;
                    f32x2 own = 0ull;   // with two accumulators the full batch took 140 us in place of 136
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int at = 8 * sub + 64 * j;
                        const auto put = [&](unsigned char *to_hi, unsigned char *to_lo, uint32_t to, const f32x2 (&x)[4]) {
                            uint32_t hi[4], lo[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) split2(unpack2(x[i]).x, unpack2(x[i]).y, hi[i], lo[i]);
                            *reinterpret_cast<uint4 *>(to_hi + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                            *reinterpret_cast<uint4 *>(to_lo + to) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        };
                        float kk[8], y[8];
                        f32x2 x[4];
                        rk[j].get(kk);
                        rb[j].get(y);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[i] = mul2(mul2(pack2(y[2 * i], y[2 * i + 1]), pack2(kk[2 * i], kk[2 * i + 1])), G[2 * j + (i >> 1)][i & 1]);
                        put(sh.b_hi, sh.b_lo, sw_off(node, at, 2 * MAX_NODES), x);
                        rq[j].get(y);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            own = fma2(pack2(y[2 * i], y[2 * i + 1]), pack2(kk[2 * i], kk[2 * i + 1]), own);
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] = mul2(pack2(y[2 * i], y[2 * i + 1]), G[2 * j + (i >> 1)][i & 1]);
                        put(sh.b_hi, sh.b_lo, sw_off(rows + node, at, 2 * MAX_NODES), x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 d = unpack2(G[2 * j + (i >> 1)][i & 1]);
                            x[i] = mul2(pack2(kk[2 * i], kk[2 * i + 1]), pack2(inverse(d.x), inverse(d.y)));
                        }
                        put(sh.k_hi, sh.k_lo, sw_off(node, at, MAX_NODES), x);
                    }
                    const float2 both = unpack2(own);
                    float sum = both.x + both.y;
#pragma unroll
                    for (int h = 4; h > 0; h >>= 1) sum += __shfl_xor_sync(0xffu << (lane & 24), sum, h);
                    if (sub == 0) sh.own[c & 1][node] = sum;
                }
                fence_async_smem();
                arrive(sh.b_full);
                ++c;
            }
            arrive(sh.meta_free[it % METAS]);
        }
    } else {
        constexpr int THREADS = 32 * PAIR_WARPS;
        const int t = tid - 32 * PAIR0;
        for (int it = 0;; ++it) {
            if (blockIdx.x + (long long)it * gridDim.x >= items) break;
            if (!group_wait(sh.meta_full[it % METAS], it / METAS, BAR_PAIR, THREADS)) break;   // paths and order too
            const Meta &m = sh.meta[it % METAS];
            const int n = m.n, rows = (n + 7) / 8 * 8;
            if (n > 0) {
                if (t < n) {
                    unsigned long long path = 0ull;
                    for (int h = 0; h <= m.above[t]; h += 4) {
                        const uchar4 a4 = *reinterpret_cast<const uchar4 *>(m.anc + pairs(t) + h);
                        path |= 1ull << a4.x | 1ull << a4.y | 1ull << a4.z | 1ull << a4.w;
                    }
                    sh.path[t] = path;
                }
                if (!group_wait(sh.coef_free[c & 1], (c >> 1) + 1, BAR_PAIR, THREADS) ||
                    !group_wait(sh.p_full, c, BAR_PAIR, THREADS))
                    break;
                float *coef = sh.c[c & 1];
                const unsigned long long fine = __ballot_sync(0xffffffffu, lane < n && m.fine[lane]) |
                                                (unsigned long long)__ballot_sync(0xffffffffu, lane + 32 < n && m.fine[lane + 32]) << 32;
                // A row a thread, half its columns: those on the row's path, where all their G are in range.  The
                // ancestor i of a node stands above(node) - above(i) places behind it.
                const int i0 = 32 * (warp - PAIR0 >> 2), line = 32 * (warp & 3) + lane, who = line < rows ? line : line - rows;
                if (i0 < n && 32 * (warp & 3) < 2 * rows) {
                    uint32_t y[32];
                    tmem_ld32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + TM_P + i0, y);
                    const unsigned long long path = who < n ? sh.path[who] : 0ull;
                    const uint32_t mine = path & ~fine ? 0u : (uint32_t)((path & ~(1ull << (who & 63))) >> i0);
                    float *to = (line < rows ? sh.a : coef) + (who < n ? pairs(who) + m.above[who] : 0);
                    wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const uchar4 a4 = *reinterpret_cast<const uchar4 *>(m.above + i0 + i);
                        if (mine >> i & 1) to[-a4.x] = __uint_as_float(y[i]);
                        if (mine >> (i + 1) & 1) to[-a4.y] = __uint_as_float(y[i + 1]);
                        if (mine >> (i + 2) & 1) to[-a4.z] = __uint_as_float(y[i + 2]);
                        if (mine >> (i + 3) & 1) to[-a4.w] = __uint_as_float(y[i + 3]);
                    }
                }
                if (t < n) coef[pairs(t)] = sh.own[c & 1][t];
                fence_before();
                arrive(sh.p_free);
                // the others from the tokens
#pragma unroll 1
                for (int round = 0; round < 2; ++round) {
                    const int node = 32 * round + (t >> 3);
                    const bool far = node < n && (sh.path[node] & ~fine);
                    if (__any_sync(0xffffffffu, far))
                        couple_far<__nv_bfloat16, D>(q, k, b, alpha, m.anc, sh.a, coef, far, m.lo, H, m.head, far ? node : 0,
                                                     far ? m.above[node] : -1, lane);
                }
                group_sync(BAR_PAIR, THREADS);   // every A and P is there
#pragma unroll 1
                for (int round = 0; round < 2; ++round) {
                    const int place = place_of(round, t >> 3);
                    const bool go = place < n;
                    if (__all_sync(0xffffffffu, !go)) continue;
                    const int node = go ? m.order[place] : 0;
                    eliminate(sh.a, coef, m.anc, coef, go, node, go ? m.above[node] : -1, lane);
                }
                arrive(sh.coef_full[c & 1]);
                ++c;
            }
            arrive(sh.meta_free[it % METAS]);
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == LEAD) {
        if (lane == 0 && *abort) atomicOr(status, DEV_WAIT);
        tmem_dealloc(tmem, TM_COLS);
    }
}

int launch_tc(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
              const float *S, long long slot_stride, int num_slots, const int *slots, const int *cu, const int *parents,
              void *o, int batch, int H, int total, int max_nodes, unsigned *status, cudaStream_t st) {
    constexpr int smem = (int)sizeof(TcShared) + 1024;
    if (!allow_smem(tree_tc_kernel, smem)) return -6;
    using bf = __nv_bfloat16;
    const long long items = (long long)batch * H;
    return launch_close(tree_tc_kernel, (unsigned)(items < 148 ? items : 148), TC_THREADS, smem, st, (const bf *)q, (const bf *)k,
                        (const bf *)v, alpha, (const bf *)b, (const bf *)w, S, slot_stride, num_slots, slots, cu, parents,
                        (bf *)o, batch, H, total, max_nodes, wait_limit(WAIT_LIMIT), status);
}

}  // namespace tree
}  // namespace gdn2
