// Drafted trees over a state cache on the tensor cores (sm_100a): bf16 tokens, d_k = d_v = 128.  The formulas are
// those of gdn2_tree.cu; what is different is where the two products with the state run, and that a
// persistent CTA's warps work on several (sequence, head) items at once.
//
// S^T [e G; q G]^T, 128 x 128 x 2n, is 2 n 128^2 FMA a head, more than CUDA cores do in the time that HBM takes
// for the state and the tokens from five nodes on.  Both factors are split into two bf16, x = hi + lo (16
// significant bits, relative error 2^-17): three tcgen05 products hi hi + hi lo + lo hi keep the error far
// below the rounding of the bf16 output, where one product of bf16 operands would double that rounding.
//   state group  (4 warps)  a column of S a thread, split, into tensor memory: the A operand S^T, lane = value
//                           column, two buffers
//   path group   (8 warps)  eight lanes a node up to its root: the rows e G and q G, split, into the B operand's
//                           swizzled images, and k / G
//   pair group   (8 warps)  the coefficients along the paths, from those
//   column group (8 warps)  R = u - S^T (e G) and S^T (q G) from tensor memory (lane = value column) to shared
//                           memory, then o = S^T (q G) + C R, two nodes a warp and eight columns a lane
//   lead warp               reads and checks the items, lists their paths, brings the tokens' lines into L2 ahead
//                           of the groups, and issues the products
#include "gdn2_tree.cuh"
#include "tc_ptx.cuh"

namespace gdn2 {
namespace tree {

using namespace gdn2::tc;

constexpr int D = 128;
constexpr int COLUMN_WARPS = 8, STATE_WARPS = 4, PATH_WARPS = 8, PAIR_WARPS = 8;   // in this order; then the lead
constexpr int PATH0 = COLUMN_WARPS + STATE_WARPS, PAIR0 = PATH0 + PATH_WARPS, LEAD = PAIR0 + PAIR_WARPS,
              TC_THREADS = 32 * (LEAD + 1);
constexpr int METAS = 3;
constexpr uint32_t BAR_COLUMN = 1, BAR_PATH = 2, BAR_PAIR = 3, BAR_STATE = 4, WAIT_LIMIT = 1u << 20;
constexpr uint32_t TM_S = 0, TM_D = 256, TM_COLS = 512;   // S: two buffers of hi (64 columns) and lo (64)

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
    float alpha[MAX_NODES][D], key[MAX_NODES][D];   // key: k / G
    float r[MAX_NODES][D], x[MAX_NODES][D];   // u, then R; S^T (q G); by node and value column
    float a[MAX_PAIRS], c[2][MAX_PAIRS];      // A; P, then C
    Meta meta[METAS];
    unsigned long long meta_full[METAS], meta_free[METAS], s_full[2], s_free[2], coef_full[2], coef_free[2], b_full, b_free,
        d_full, d_free;
    uint32_t tmem, abort;
};
static_assert(sizeof(TcShared) + 1024 <= 227 * 1024, "shared memory of an SM");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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
    int total, int max_nodes, unsigned *status) {
    extern __shared__ unsigned char raw[];
    TcShared &sh = *reinterpret_cast<TcShared *>(raw + ((1024 - (smem_u32(raw) & 1023)) & 1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long items = (long long)batch * H;
    const auto bar = [](unsigned long long &x) { return smem_u32(&x); };
    volatile uint32_t *abort = &sh.abort;

    if (tid == 0) {
        for (int i = 0; i < METAS; ++i) mbar_init(bar(sh.meta_full[i]), 1), mbar_init(bar(sh.meta_free[i]), LEAD);   // a warp each, but the lead
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(sh.s_full[i]), STATE_WARPS);
            mbar_init(bar(sh.s_free[i]), 1);
            mbar_init(bar(sh.coef_full[i]), PAIR_WARPS);
            mbar_init(bar(sh.coef_free[i]), COLUMN_WARPS);
        }
        mbar_init(bar(sh.b_full), PATH_WARPS);
        mbar_init(bar(sh.b_free), 1 + PAIR_WARPS);   // the products, and the pair group
        mbar_init(bar(sh.d_full), 1);
        mbar_init(bar(sh.d_free), COLUMN_WARPS);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == LEAD) tmem_alloc(smem_u32(&sh.tmem), TM_COLS);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem;

    // Every wait is bounded, and every thread of a group gets the same verdict, so that none is left at one of
    // the group's barriers.  One warp of a group polls, the others sleep at the barrier.  Phases count the items
    // that have nodes (c); the others only pass their meta on.
    const auto wait = [&](unsigned long long &x, int phase) {
        const bool ok = mbar_wait(bar(x), phase & 1, WAIT_LIMIT) && !*abort;
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
    if (warp == LEAD) {
        const auto look = [&](long long at, Meta &m) {
            const int seq = (int)(at / H), head = (int)(at % H), lo = cu[seq], hi = cu[seq + 1], slot = slots[seq];
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
            __syncwarp();
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
            __syncwarp();
            return n;
        };
        int before = 0;   // nodes of the item before
        for (int it = 0;; ++it) {
            const long long at = blockIdx.x + (long long)it * gridDim.x;
            int n = 0;
            if (at < items) {
                if (!warp_wait(sh.meta_free[it % METAS], it / METAS + 1)) break;
                n = look(at, sh.meta[it % METAS]);
                arrive(sh.meta_full[it % METAS]);
            }
            if (before > 0) {   // the item before: its products
                const int rows = (before + 7) / 8 * 8;
                if (!warp_wait(sh.s_full[c & 1], c >> 1) || !warp_wait(sh.b_full, c) || !warp_wait(sh.d_free, c + 1)) break;
                fence_after();
                if (lane == 0) {
                    const uint32_t idesc = idesc_bf16(128, 2 * rows, 0, 0), s = tmem + TM_S + (c & 1) * 128;
                    const auto products = [&](uint32_t a, uint64_t desc, uint32_t acc) {   // eight steps of 16 channels
#pragma unroll
                        for (int j = 0; j < 8; ++j)   // the address field counts 16 bytes: 32 bytes a step, 16 KB a half
                            mma_ts(tmem + TM_D, a + 8 * j, desc + (j >> 2) * (2 * MAX_NODES * 128 >> 4) + (j & 3) * 2, idesc, acc | (j > 0));
                    };
                    const uint64_t hi = desc_kmajor(smem_u32(sh.b_hi), 2 * MAX_NODES, 0),
                                   lo = desc_kmajor(smem_u32(sh.b_lo), 2 * MAX_NODES, 0);
                    products(s, hi, 0);
                    products(s, lo, 1);
                    products(s + 64, hi, 1);
                    mma_commit(bar(sh.s_free[c & 1]));
                    mma_commit(bar(sh.b_free));
                    mma_commit(bar(sh.d_full));
                }
                __syncwarp();
                ++c;
            }
            if (at >= items) break;
            before = n;
        }
    } else if (warp < COLUMN_WARPS) {
        const int col = tid & 127, half = tid >> 7;   // value column, warpgroup
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        for (int it = 0;; ++it) {
            if (blockIdx.x + (long long)it * gridDim.x >= items) break;
            if (!group_wait(sh.meta_full[it % METAS], it / METAS, BAR_COLUMN, 32 * COLUMN_WARPS)) break;
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
            if (!group_wait(sh.meta_full[it % METAS], it / METAS, BAR_STATE, 32 * STATE_WARPS)) break;
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
            if (!group_wait(sh.meta_full[it % METAS], it / METAS, BAR_PATH, THREADS)) break;   // and the last item's climbs
            Meta &m = sh.meta[it % METAS];
            const int n = m.n, rows = (n + 7) / 8 * 8;
            if (n > 0) {
                const size_t first = ((size_t)m.lo * H + m.head) * D;
                for (int i = t; i < n * (D / 4); i += THREADS)
                    cp_async16(smem_u32(&sh.alpha[0][0]) + 16 * i, alpha + first + (size_t)(i / (D / 4)) * H * D + i % (D / 4) * 4);
                bool ok = true;
#pragma unroll 1
                for (int round = 0; round < 2; ++round) {
                    const int place = place_of(round, t >> 3);
                    const bool go = place < n;
                    const int node = go ? m.order[place] : 0, above = go ? m.above[node] : -1;
                    Raw<__nv_bfloat16, 4> rk[4], rb[4], rq[4];
                    const size_t row = first + (size_t)node * H * D + 4 * sub;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        rk[j].clear();
                        rb[j].clear();
                        rq[j].clear();
                        if (go) rk[j].load(k + row + 32 * j), rb[j].load(b + row + 32 * j), rq[j].load(q + row + 32 * j);
                    }
                    if (round == 0) {
                        cp_async_wait();
                        group_sync(BAR_PATH, THREADS);
                    }
                    f32x2 G[4][2];
                    climb<D>(&sh.alpha[0][0], m.anc, go, node, above, lane, G);
                    const bool good = in_range<D>(G, lane);
                    // the products and the pairs of the item before
                    if (round == 0 && !(ok = group_wait(sh.b_free, c + 1, BAR_PATH, THREADS))) break;
                    if (!go) continue;
                    if (sub == 0) m.fine[node] = good;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float kk[4], bb[4], qq[4];
                        rk[j].get(kk);
                        rb[j].get(bb);
                        rq[j].get(qq);
                        const float2 g0 = unpack2(G[j][0]), g1 = unpack2(G[j][1]);
                        *reinterpret_cast<float4 *>(&sh.key[node][4 * (sub + 8 * j)]) =
                            make_float4(kk[0] * inverse(g0.x), kk[1] * inverse(g0.y), kk[2] * inverse(g1.x), kk[3] * inverse(g1.y));
                        const auto put = [&](int to, f32x2 x, f32x2 y) {
                            const float2 x0 = unpack2(x), x1 = unpack2(y);
                            const uint32_t at = sw_off(to, 4 * (sub + 8 * j), 2 * MAX_NODES);
                            uint2 hi, lo2;
                            split2(x0.x, x0.y, hi.x, lo2.x);
                            split2(x1.x, x1.y, hi.y, lo2.y);
                            *reinterpret_cast<uint2 *>(sh.b_hi + at) = hi;
                            *reinterpret_cast<uint2 *>(sh.b_lo + at) = lo2;
                        };
                        put(node, mul2(mul2(pack2(bb[0], bb[1]), pack2(kk[0], kk[1])), G[j][0]),
                            mul2(mul2(pack2(bb[2], bb[3]), pack2(kk[2], kk[3])), G[j][1]));
                        put(rows + node, mul2(pack2(qq[0], qq[1]), G[j][0]), mul2(pack2(qq[2], qq[3]), G[j][1]));
                    }
                }
                if (!ok) break;
                fence_async_smem();
                arrive(sh.b_full);
                ++c;
            }
            arrive(sh.meta_free[it % METAS]);
        }
    } else {
        constexpr int THREADS = 32 * PAIR_WARPS;
        const int t = tid - 32 * PAIR0, sub = lane & 7;
        for (int it = 0;; ++it) {
            if (blockIdx.x + (long long)it * gridDim.x >= items) break;
            if (!group_wait(sh.meta_full[it % METAS], it / METAS, BAR_PAIR, THREADS)) break;
            const Meta &m = sh.meta[it % METAS];
            const int n = m.n, rows = (n + 7) / 8 * 8;
            if (n > 0) {
                if (!group_wait(sh.coef_free[c & 1], (c >> 1) + 1, BAR_PAIR, THREADS) ||
                    !group_wait(sh.b_full, c, BAR_PAIR, THREADS))
                    break;
                float *coef = sh.c[c & 1];
#pragma unroll 1
                for (int round = 0; round < 2; ++round) {
                    const int place = place_of(round, t >> 3);
                    const bool go = place < n;
                    if (__all_sync(0xffffffffu, !go)) continue;
                    const int node = go ? m.order[place] : 0, above = go ? m.above[node] : -1;
                    bool good = go;
                    for (int j = sub; j <= above; j += 8) good = good && m.fine[m.anc[pairs(node) + j]];
                    good = (__ballot_sync(0xffffffffu, good) >> (lane & 24) & 0xffu) == 0xffu;
                    f32x2 e[4][2], g[4][2];   // the rows again: hi + lo
                    const auto get = [&](int from, int j, f32x2 (&x)[2]) {
                        const uint32_t at = sw_off(from, 4 * (sub + 8 * j), 2 * MAX_NODES);
                        const uint2 hi = *reinterpret_cast<const uint2 *>(sh.b_hi + at), lo2 = *reinterpret_cast<const uint2 *>(sh.b_lo + at);
                        const auto two = [](uint32_t x) { return pack2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)); };
                        x[0] = add2(two(hi.x), two(lo2.x));
                        x[1] = add2(two(hi.y), two(lo2.y));
                    };
#pragma unroll
                    for (int j = 0; j < 4; ++j) get(node, j, e[j]), get(rows + node, j, g[j]);
                    couple<D>(&sh.key[0][0], m.anc, sh.a, coef, good, node, above, lane, e, g);
                    if (__any_sync(0xffffffffu, go && !good))
                        couple_far<__nv_bfloat16, D>(q, k, b, alpha, m.anc, sh.a, coef, go && !good, m.lo, H, m.head, node, above,
                                                     lane);
                }
                arrive(sh.b_free);
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
    tree_tc_kernel<<<(unsigned)(items < 148 ? items : 148), TC_THREADS, smem, st>>>(
        (const bf *)q, (const bf *)k, (const bf *)v, alpha, (const bf *)b, (const bf *)w, S, slot_stride, num_slots, slots,
        cu, parents, (bf *)o, batch, H, total, max_nodes, status);
    return launch_status();
}

}  // namespace tree
}  // namespace gdn2
