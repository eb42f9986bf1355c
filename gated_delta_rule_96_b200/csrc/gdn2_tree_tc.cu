// Drafted trees over a state cache on the tensor cores (sm_100a): bf16 tokens, d_k = d_v = 128.  The formulas are
// those of gdn2_tree.cu; what is different is where the two products with the state run, and that a
// persistent CTA's warps work on three (sequence, head) items at once.
//
// S^T [e G; q G]^T, 128 x 128 x 2n, is 2 n 128^2 FMA a head, more than CUDA cores do in the time that HBM takes
// for the state and the tokens from five nodes on.  Both factors are split into two bf16, x = hi + lo (16
// significant bits, relative error 2^-17): three tcgen05 products hi hi + hi lo + lo hi keep the error far
// below the rounding of the bf16 output, where one product of bf16 operands would double that rounding.
//   state group  (8 warps)  S from HBM to registers, half a column a thread, split, into tensor memory: the A
//                           operand S^T, lane = value column, two buffers
//   walk group   (8 warps)  eight lanes a node up to its root, then the elimination: the coefficients to shared
//                           memory, and the rows e G and q G, split, into the B operand's swizzled images
//   column group (8 warps)  R = u - S^T (e G) and S^T (q G) from tensor memory (lane = value column) to shared
//                           memory, then o = S^T (q G) + C R, a node a warp and four columns a lane
//   lead warp               reads and checks the items, brings the tokens' lines into L2 ahead of the groups,
//                           and issues the products
#include "gdn2_tree.cuh"
#include "tc_ptx.cuh"

namespace gdn2 {
namespace tree {

using namespace gdn2::tc;

constexpr int D = 128;
constexpr int COLUMN_WARPS = 8, STATE_WARPS = 8, WALK_WARPS = 8;   // in this order; then the lead warp
constexpr int LEAD = COLUMN_WARPS + STATE_WARPS + WALK_WARPS, TC_THREADS = 32 * (LEAD + 1);
constexpr int METAS = 4;
constexpr uint32_t BAR_COLUMN = 1, BAR_WALK = 2, BAR_STATE = 3, WAIT_LIMIT = 1u << 24;
constexpr uint32_t TM_S = 0, TM_D = 256, TM_COLS = 512;   // S: two buffers of hi (64 columns) and lo (64)

// An item: its nodes lo .. lo+n-1, their parents, the state's slot.
struct Meta {
    int lo, n, slot, head;
    signed char parent[MAX_NODES];
};

struct Coef {   // eliminate()'s, whom each is for, and how many ancestors a node has
    float c[MAX_PAIRS];
    unsigned char anc[MAX_PAIRS], above[MAX_NODES];
};

struct TcShared {
    unsigned char b_hi[2 * MAX_NODES * D * 2], b_lo[2 * MAX_NODES * D * 2];   // [e G; q G], swizzled
    __nv_bfloat16 k[MAX_NODES][D];
    float alpha[MAX_NODES][D];
    float r[MAX_NODES][D], x[MAX_NODES][D];   // u, then R; S^T (q G); by node and value column
    float a[MAX_PAIRS];
    unsigned short where[MAX_PAIRS];
    Coef coef[2];
    Meta meta[METAS];
    unsigned long long meta_full[METAS], meta_free[METAS], s_full[2], s_free[2], coef_full[2], coef_free[2], b_full,
        b_free, d_full, d_free;
    uint32_t tmem, abort;
};
static_assert(sizeof(TcShared) + 1024 <= 227 * 1024, "shared memory of an SM");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// x = hi + lo, two values at a time as packed bf16 (the first in the low half).  A value that is not finite
// stays in hi alone: inf - inf would put a NaN into lo.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(x, y);
    const float hx = __uint_as_float(hi << 16), hy = __uint_as_float(hi & 0xffff0000u);
    lo = pack_bf16(fabsf(hx) < INFINITY ? x - hx : 0.f, fabsf(hy) < INFINITY ? y - hy : 0.f);
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
        for (int i = 0; i < METAS; ++i) mbar_init(bar(sh.meta_full[i]), 1), mbar_init(bar(sh.meta_free[i]), LEAD);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(sh.s_full[i]), STATE_WARPS);
            mbar_init(bar(sh.s_free[i]), 1);
            mbar_init(bar(sh.coef_full[i]), WALK_WARPS);
            mbar_init(bar(sh.coef_free[i]), COLUMN_WARPS);
        }
        mbar_init(bar(sh.b_full), WALK_WARPS);
        mbar_init(bar(sh.b_free), 1);
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
    const auto group_wait = [&](unsigned long long &x, int phase, uint32_t id) {
        const bool polls = (warp & 7) == 0, ok = !group_or(id, 256, polls && !wait(x, phase));
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
            if (!group_wait(sh.meta_full[it % METAS], it / METAS, BAR_COLUMN)) break;
            const Meta &m = sh.meta[it % METAS];
            const int n = m.n;
            if (n > 0) {
                const size_t first = ((size_t)m.lo * H + m.head) * D;
                // u, eight columns a thread at a time (group_wait's barrier is behind the last item's reads)
#pragma unroll 4
                for (int i = tid; i < n * (D / 8); i += 256) {
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
                if (!group_wait(sh.d_full, c, BAR_COLUMN)) break;
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
                if (!group_wait(sh.coef_full[c & 1], c >> 1, BAR_COLUMN)) break;
                const Coef &coef = sh.coef[c & 1];
                for (int node = warp; node < n; node += COLUMN_WARPS) {   // four columns a lane
                    const int base = pairs(node), above = coef.above[node];
                    f32x2 x[2];
                    load2(&sh.x[node][4 * lane], x);
                    for (int j = 0; j <= above; j += 4) {
                        const float4 c4 = *reinterpret_cast<const float4 *>(coef.c + base + j);
                        const uchar4 a4 = *reinterpret_cast<const uchar4 *>(coef.anc + base + j);
                        const float cc[4] = {c4.x, c4.y, c4.z, c4.w};
                        const int from[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            f32x2 r[2];
                            load2(&sh.r[from[i]][4 * lane], r);
                            x[0] = fma2(pack2(cc[i], cc[i]), r[0], x[0]);
                            x[1] = fma2(pack2(cc[i], cc[i]), r[1], x[1]);
                        }
                    }
                    const float2 x0 = unpack2(x[0]), x1 = unpack2(x[1]);
                    *reinterpret_cast<uint2 *>(o + first + (size_t)node * H * D + 4 * lane) =
                        make_uint2(pack_bf16(x0.x, x0.y), pack_bf16(x1.x, x1.y));
                }
                arrive(sh.coef_free[c & 1]);
                ++c;
            }
            arrive(sh.meta_free[it % METAS]);
        }
    } else if (warp < COLUMN_WARPS + STATE_WARPS) {
        const int col = tid & 127, half = (warp - COLUMN_WARPS) >> 2;   // rows 64 half .. of the state
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        for (int it = 0;; ++it) {
            if (blockIdx.x + (long long)it * gridDim.x >= items) break;
            if (!group_wait(sh.meta_full[it % METAS], it / METAS, BAR_STATE)) break;
            const Meta &m = sh.meta[it % METAS];
            const int n = m.n, slot = m.slot, head = m.head;
            arrive(sh.meta_free[it % METAS]);
            if (n == 0) continue;
            const float *src = S + (size_t)(slot < 0 ? 0 : slot) * slot_stride + ((size_t)head * D + 64 * half) * D + col;
            const uint32_t to = tmem + lanes + TM_S + (c & 1) * 128 + 32 * half;
            bool ok = true;
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                float x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = slot < 0 ? 0.f : __ldcs(src + (size_t)(32 * part + i) * D);
                if (part == 0) {
                    if (!(ok = group_wait(sh.s_free[c & 1], (c >> 1) + 1, BAR_STATE))) break;
                }
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
    } else {
        const int t = tid - 32 * (COLUMN_WARPS + STATE_WARPS), ww = t >> 5, sub = lane & 7;
        for (int it = 0;; ++it) {
            if (blockIdx.x + (long long)it * gridDim.x >= items) break;
            if (!group_wait(sh.meta_full[it % METAS], it / METAS, BAR_WALK)) break;
            const Meta &m = sh.meta[it % METAS];
            const int n = m.n;
            if (n > 0) {
                const int lo = m.lo, head = m.head, rows = (n + 7) / 8 * 8;
                const size_t first = ((size_t)lo * H + head) * D;
                for (int i = t; i < n * (D / 4); i += 256) {   // group_wait's barrier is behind the last walk
                    const int node = i / (D / 4), at = i % (D / 4) * 4;
                    cp_async16(smem_u32(&sh.alpha[node][at]), alpha + first + (size_t)node * H * D + at);
                    if (!(i & 1)) cp_async16(smem_u32(&sh.k[node][at]), k + first + (size_t)node * H * D + at);
                }
                // the second half from the other end: late nodes are deep, and a warp has both
                const int node_of[2] = {4 * ww + (lane >> 3), 63 - 4 * ww - (lane >> 3)};
                Rows<__nv_bfloat16, D> tok;
                tok.load(b, q, lo, H, head, node_of[0], n, lane);
                cp_async_wait();
                if (!group_wait(sh.coef_free[c & 1], (c >> 1) + 1, BAR_WALK)) break;
                Coef &coef = sh.coef[c & 1];
                bool ok = true;
#pragma unroll 1
                for (int round = 0; round < 2; ++round) {
                    if (32 * round >= n) break;
                    const int node = round ? node_of[1] : node_of[0];
                    f32x2 e[4][2], g[4][2];
                    const int up = walk<__nv_bfloat16, D>(tok, &sh.k[0][0], &sh.alpha[0][0], m.parent, sh.a, coef.c, coef.anc,
                                                          sh.where, node, n, lane, e, g);
                    if (round == 0) {
                        if (!(ok = group_wait(sh.b_free, c + 1, BAR_WALK))) break;   // the products before
                        if (n > 32) tok.load(b, q, lo, H, head, node_of[1], n, lane);
                    }
                    if (node < n) {
                        if (sub == 0) coef.above[node] = (unsigned char)up;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t at = sw_off(node, 4 * (sub + 8 * j), 2 * MAX_NODES),
                                           at2 = sw_off(rows + node, 4 * (sub + 8 * j), 2 * MAX_NODES);
                            const auto put = [&](uint32_t to, const f32x2 (&x)[2]) {
                                const float2 x0 = unpack2(x[0]), x1 = unpack2(x[1]);
                                uint2 hi, lo2;
                                split2(x0.x, x0.y, hi.x, lo2.x);
                                split2(x1.x, x1.y, hi.y, lo2.y);
                                *reinterpret_cast<uint2 *>(sh.b_hi + to) = hi;
                                *reinterpret_cast<uint2 *>(sh.b_lo + to) = lo2;
                            };
                            put(at, e[j]);
                            put(at2, g[j]);
                        }
                    }
                }
                if (!ok) break;
                fence_async_smem();
                arrive(sh.b_full);
                group_sync(BAR_WALK, 256);   // every walk is done
#pragma unroll 1
                for (int round = 0; round < 2; ++round) {
                    const int node = round ? node_of[1] : node_of[0];
                    if (32 * round >= n) break;
                    eliminate(sh.a, coef.c, sh.where, coef.c, node, n, node < n ? coef.above[node] : 0, lane);
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
    static const bool ok =
        cudaFuncSetAttribute(tree_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess;
    if (!ok) return -6;
    using bf = __nv_bfloat16;
    const long long items = (long long)batch * H;
    tree_tc_kernel<<<(unsigned)(items < 148 ? items : 148), TC_THREADS, smem, st>>>(
        (const bf *)q, (const bf *)k, (const bf *)v, alpha, (const bf *)b, (const bf *)w, S, slot_stride, num_slots, slots,
        cu, parents, (bf *)o, batch, H, total, max_nodes, status);
    return launch_status();
}

}  // namespace tree
}  // namespace gdn2
