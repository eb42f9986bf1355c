// The recurrence over slots of a state cache, for ragged runs of tokens (sm_100a; page "NVIDIA представила
// Gated DeltaNet-2 ...", section "Техническая схема", the state-update equation).
//
// Sequence i owns the tokens cu[i] .. cu[i+1]-1 (through `index`, if given); its state is read from slot
// slots_in[i] and written to slot slots_out[i].  Four tokens at a time in the chunk form, with G_t the product
// of the block's decays up to t (its own included), e = b k, u = w v:
//   delta_t = u_t - S^T (e_t G_t) - sum_{i<t} A[t,i] delta_i,   A[t,i] = sum_c e_t (G_t / G_i) k_i
//   o_t     = S^T (q_t G_t) + sum_{i<=t} P[t,i] delta_i,        P[t,i] = sum_c q_t (G_t / G_i) k_i
//   S      <- Diag(G_3) S + sum_t (k_t G_3 / G_t) delta_t^T
// which takes 13 FMA for each element of S where the recurrence takes 16, and one chain of reductions in
// place of four.  The ratios of G are running products of decays, never quotients, so any decay is exact.
// Everything is fp32: the states are returned in it and go on to the next call.
//
// The columns of S are independent of one another: a consumer warp owns 16 of them from the first token to
// the last, lane = (row group rg = lane >> 2, column group lane & 3), rows 4 (rg + 8 j) + i, four columns, which
// keeps its slice of the state in K/2 registers a lane.  One CTA an SM walks the (sequence, head, column
// range) items, and every latency but the arithmetic is another warp's:
//   scout      reads an item's lengths and slots, checks them, and has a bulk copy bring its state into one of
//              DEPTH buffers, an item ahead;
//   producers  turn the tokens into the block's vectors and coefficients, up to RING blocks ahead;
//   consumers  state to registers, the blocks, state back to the buffer;
//   storer     has a bulk copy take the buffer to the slot, and frees it once it has been read.
// Where a head's columns are split over CTAs (few chains), the consumers move their own part of the state.
// A decode step (one token, 128 KB moved for 0.1 MFMA a head) is then bound by HBM: B256 H16 d128 takes 90 us, 6.0
// of the 6.5 TB/s that a plain copy reaches; with the state loaded to registers by two CTAs an SM, which each
// waited for every latency in turn, it took 166.  Accepted paths (B64 H16 d128, up to 9 tokens) take 43 us, twice
// their 145 MB: there it is the consumers, 3,200 cycles for a block of four tokens, as many issue slots for LDS as for
// FMA, and 2,500 to move a state between shared memory and registers.  fp32 runs of up to 201 tokens (B8 H16 d64) take
// 46 us, the longest chain's 1,400 cycles a block, one after the other (d128, in bf16 and in fp32: 99 us).
#include <atomic>

#include "gdn2_internal.h"
#include "gdn2_slots.cuh"
#include "tc_ptx.cuh"

namespace gdn2 {
namespace rec {

using namespace gdn2::tc;

constexpr int M = 4;           // tokens of a block
// producer warps: each takes about 4,000 cycles for a block, most of it latency; where the consumers of a
// whole head take longer for two, two are enough and leave them 168 registers a thread
template <int K, int V>
constexpr int PRODUCERS = K == 128 && V == 128 ? 2 : 4;
constexpr int DEPTH = 2;       // state buffers: one worked on, one on its way in or out
constexpr int RING = 6;        // token blocks ahead
// Limits of the waits, in polls.  A poll that finds nothing sleeps for some 4 us (runs of 20,000 and 100,000 tokens), so
// WAIT_LIMIT is 8 s.  The storer and the scout wait for a whole run, measured 0.13 to 0.4 us a token: 4 polls a token,
// 16 us, are added for it.
constexpr uint32_t WAIT_LIMIT = 1u << 21, WAIT_TOKEN = 4;

template <int K, int V>
struct Block {
    float e[M][K], q[M][K], k[M][K], g[K];   // e G, q G, k G_3 / G, G_3
    float u[M][V];                           // w v (the columns of this CTA)
    float coef[16];                          // A10 A20 A21 A30 A31 A32, P00 P10 P11 P20 .. P33
};

template <int CPL>
__device__ __forceinline__ void store_f32(float *p, const float (&x)[CPL]) {
    if constexpr (CPL == 4) *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
}

// A producer warp's work on one block: up to M tokens (the missing ones are neutral: decay 1, the rest 0).
template <typename Tok, int K, int V>
__device__ __forceinline__ void produce(Block<K, V> &out, const Tok *q, const Tok *k, const Tok *v, const float *alpha,
                                        const Tok *b, const Tok *w, const int *index, int t0, int n, int H, int head,
                                        int col0, int cols, int lane) {
    constexpr int CPL = K / 32;
    // every load before the first store: one latency for the block
    Raw<float, CPL> ra[M];
    Raw<Tok, CPL> rk[M], rb[M], rq[M];   // kept as stored until a token's turn: registers
    Raw<Tok, 4> rv[M], rw[M];
    int token[M];
#pragma unroll
    for (int t = 0; t < M; ++t) token[t] = t < n ? (index ? index[t0 + t] : t0 + t) : -1;
#pragma unroll
    for (int t = 0; t < M; ++t) {
        rk[t].clear();
        rb[t].clear();
        rq[t].clear();
        rv[t].clear();
        rw[t].clear();
#pragma unroll
        for (int c = 0; c < CPL; ++c) ra[t].r[c] = __float_as_uint(1.f);
        if (t < n) {
            const size_t row = (size_t)token[t] * H + head;
            ra[t].load(alpha + row * K + lane * CPL);
            rk[t].load(k + row * K + lane * CPL);
            rb[t].load(b + row * K + lane * CPL);
            rq[t].load(q + row * K + lane * CPL);
            if (lane * 4 < cols) {
                rv[t].load(v + row * V + col0 + lane * 4);
                rw[t].load(w + row * V + col0 + lane * 4);
            }
        }
    }
    float a[M][CPL];
#pragma unroll
    for (int t = 0; t < M; ++t) {
        ra[t].get(a[t]);
        float vv[4], ww[4];
        rv[t].get(vv);
        rw[t].get(ww);
#pragma unroll
        for (int c = 0; c < 4; ++c) vv[c] *= ww[c];
        if (lane * 4 < cols) store_f32<4>(&out.u[t][lane * 4], vv);
    }
    float x[16];
#pragma unroll
    for (int t = 0; t < M; ++t) {   // from t back to the block's first token with a running product of decays
        const int A0 = t * (t - 1) / 2, P0 = 6 + t * (t + 1) / 2;
        float e[CPL], qq[CPL], kk[CPL];
        rk[t].get(kk);
        rb[t].get(e);
        rq[t].get(qq);
        x[P0 + t] = 0.f;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            x[P0 + t] = fmaf(qq[c], kk[c], x[P0 + t]);
            e[c] *= kk[c] * a[t][c];
            qq[c] *= a[t][c];
        }
#pragma unroll
        for (int i = t - 1; i >= 0; --i) {
            rk[i].get(kk);
            x[A0 + i] = x[P0 + i] = 0.f;
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                x[A0 + i] = fmaf(e[c], kk[c], x[A0 + i]);
                x[P0 + i] = fmaf(qq[c], kk[c], x[P0 + i]);
                e[c] *= a[i][c];
                qq[c] *= a[i][c];
            }
        }
        store_f32<CPL>(&out.e[t][lane * CPL], e);
        store_f32<CPL>(&out.q[t][lane * CPL], qq);
    }
    float g[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) g[c] = 1.f;
#pragma unroll
    for (int t = M - 1; t >= 0; --t) {
        float kk[CPL];
        rk[t].get(kk);
#pragma unroll
        for (int c = 0; c < CPL; ++c) kk[c] *= g[c], g[c] *= a[t][c];
        store_f32<CPL>(&out.k[t][lane * CPL], kk);
    }
    store_f32<CPL>(&out.g[lane * CPL], g);
    // sums of the sixteen values over the lanes: each step halves the values a lane carries
#pragma unroll
    for (int h = 8, m = 16; h > 0; h /= 2, m /= 2) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < h; ++i)
            x[i] = (up ? x[i + h] : x[i]) + __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + h], m);
    }
    x[0] += __shfl_xor_sync(0xffffffffu, x[0], 1);
    if (!(lane & 1)) out.coef[lane >> 1] = x[0];
}

// Sums over the 8 row groups of N tokens x 4 columns (x[4 t + c]): on return x[t] is the total of token t at
// the lane's column lane >> 3 of its four.
template <int N>
__device__ __forceinline__ void column_sums(float (&x)[4 * N], int lane) {
    const bool hi = lane & 16, lo = lane & 8;
#pragma unroll
    for (int t = 0; t < N; ++t) {
        const float a = (hi ? x[4 * t + 2] : x[4 * t]) + __shfl_xor_sync(0xffffffffu, hi ? x[4 * t] : x[4 * t + 2], 16);
        const float b = (hi ? x[4 * t + 3] : x[4 * t + 1]) + __shfl_xor_sync(0xffffffffu, hi ? x[4 * t + 1] : x[4 * t + 3], 16);
        const float s = (lo ? b : a) + __shfl_xor_sync(0xffffffffu, lo ? a : b, 8);
        x[t] = s + __shfl_xor_sync(0xffffffffu, s, 4);
    }
}

// A consumer warp's step over the first n of a block's tokens, as N >= n tokens (the others are neutral).
// Straight-line code (whether o is wanted is known to the compiler): the products with q fill the latency of
// the sums over the lanes and of the substitution.
template <typename Tok, int K, int V, int N, bool OUT>
__device__ __forceinline__ void consume(const Block<K, V> &in, float (&s)[K / 32][4][4], Tok *o, int t0, int n, int H,
                                        int head, int col0, int local, int lane) {
    constexpr int RJ = K / 32, GROUP = K == 64 || N == 1 ? N : 2;   // tokens at a time: registers
    const int rg = lane >> 2, mine = local + (lane & 3) * 4 + (lane >> 3);   // the lane's column, within the CTA's
    float e[N], q[N], d[N];   // S^T (e G), S^T (q G) of the lane's column
    auto products = [&](const float (&vec)[M][K], float (&out)[N]) {
#pragma unroll
        for (int h = 0; h < N; h += GROUP) {
            float p[4 * GROUP];
#pragma unroll
            for (int i = 0; i < 4 * GROUP; ++i) p[i] = 0.f;
#pragma unroll
            for (int j = 0; j < RJ; ++j)
#pragma unroll
                for (int t = 0; t < GROUP; ++t) {
                    const float4 x4 = *reinterpret_cast<const float4 *>(&vec[h + t][4 * (rg + 8 * j)]);
                    const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < 4; ++c) p[4 * t + c] = fmaf(x[i], s[j][i][c], p[4 * t + c]);
                }
            column_sums<GROUP>(p, lane);
#pragma unroll
            for (int t = 0; t < GROUP; ++t) out[h + t] = p[t];
        }
    };
    products(in.e, e);
    if constexpr (OUT) products(in.q, q);
#pragma unroll
    for (int t = 0; t < N; ++t) {
        d[t] = in.u[t][mine] - e[t];
#pragma unroll
        for (int i = 0; i < t; ++i) d[t] = fmaf(-in.coef[t * (t - 1) / 2 + i], d[i], d[t]);
    }
    asm volatile("" ::: "memory");   // the loads below stay below: registers
#pragma unroll
    for (int j = 0; j < RJ; ++j) {
        const float4 g4 = *reinterpret_cast<const float4 *>(&in.g[4 * (rg + 8 * j)]);
        const float g[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[j][i][c] *= g[i];
    }
#pragma unroll
    for (int t = 0; t < N; ++t) {
        float dd[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) dd[c] = __shfl_sync(0xffffffffu, d[t], (lane & 3) | (8 * c));
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
            const float4 k4 = *reinterpret_cast<const float4 *>(&in.k[t][4 * (rg + 8 * j)]);
            const float kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[j][i][c] = fmaf(kk[i], dd[c], s[j][i][c]);
        }
    }
    if constexpr (OUT) {
#pragma unroll
        for (int t = 0; t < N; ++t) {
#pragma unroll
            for (int i = 0; i <= t; ++i) q[t] = fmaf(in.coef[6 + t * (t + 1) / 2 + i], d[i], q[t]);
            if (t < n && (t & 1) == (rg & 1)) store_tok(o + ((size_t)(t0 + t) * H + head) * V + col0 + mine, q[t]);
        }
    }
}

// An item as the scout found it; a malformed one, and one with nothing to do, has n = 0, from = to = -1.
// The divisions that give its head and column range are the scout's, ahead of the others.
struct Item {
    int lo, n, from, to, head, col0;
};

template <int K, int V>
struct Shared {
    Block<K, V> ring[RING];
    Item item[DEPTH];
    // item: known; state: landed; done: consumers finished; read: producers and storer finished with it
    unsigned long long known[DEPTH], landed[DEPTH], done[DEPTH], read[DEPTH], full[RING], empty[RING];
};

template <int K, int V>
constexpr size_t smem_bytes(int cols) { return sizeof(Shared<K, V>) + (cols < V ? 0 : sizeof(float) * (size_t)DEPTH * K * V); }

// Conflicts between sequences.  Below TABLE_BATCH sequences the scout compares an item's destination with every sequence's
// slots, an item ahead; for more of them that takes longer than the item, and for all items it grows with the square.
// From there on a CTA first marks the slots of the call in two bit maps of up to MAX_BUCKETS (slots a multiple of that
// apart share a place): touched, and touched by more than one sequence; only what stands in the second is compared.
// Runs of one token, H16, us without / with: B16 d128 9 / 10, d64 5 / 6; B128 50 / 49, 17 / 15; B256 94 / 90, 38 / 31;
// B1024 577 / 335, 270 / 106; B4096 7,300 / 1,313, 3,075 / 407; B16384 354,000 / 5,233, 76,700 / 1,608.
constexpr int TABLE_BATCH = 128, MAX_BUCKETS = 1 << 17;
constexpr size_t table_bytes(int buckets) { return (size_t)buckets / 4; }

__device__ __forceinline__ bool by_more(const uint32_t *table, int buckets, int slot) {
    const uint32_t at = (uint32_t)slot % (uint32_t)buckets;
    return table[(buckets + at) >> 5] >> (at & 31) & 1u;
}
// By the whole block, before anything else and as a call of its own: inlined, or further down, it made the kernel spill in
// its loops (accepted paths 43 -> 50 us).
__device__ __noinline__ void mark_slots(uint32_t *table, int buckets, const int *slots_in, const int *slots_out, int batch,
                                           int num_slots) {
    const auto mark = [&](int slot) {
        if (slot < 0 || slot >= num_slots) return;
        const uint32_t at = (uint32_t)slot % (uint32_t)buckets, bit = 1u << (at & 31);
        if (atomicOr(table + (at >> 5), bit) & bit) atomicOr(table + ((buckets + at) >> 5), bit);
    };
    for (int i = threadIdx.x; i < buckets / 16; i += blockDim.x) table[i] = 0u;
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < batch; i += blockDim.x) {
        const int from = slots_in[i], to = slots_out[i];
        mark(to);
        if (from != to) mark(from);
    }
}

// warps: consumers (16 columns each), PRODUCERS, scout, storer
template <int K, int V>
constexpr int EXTRA_WARPS = PRODUCERS<K, V> + 2;

template <typename Tok, int K, int V, bool OUT>
__global__ void __launch_bounds__(2 * V + 32 * EXTRA_WARPS<K, V>) recurrent_kernel(
    const Tok *__restrict__ q, const Tok *__restrict__ k, const Tok *__restrict__ v, const float *__restrict__ alpha,
    const Tok *__restrict__ b, const Tok *__restrict__ w, float *S, long long slot_stride, int num_slots,
    const int *__restrict__ slots_in, const int *__restrict__ slots_out, const int *__restrict__ cu,
    const int *__restrict__ index, Tok *__restrict__ o, int batch, int H, int splits, int total, int rows,
    int buckets, uint32_t limit, unsigned *status) {
    constexpr int RJ = K / 32, NP = PRODUCERS<K, V>;
    // a producer waits for a ring slot's last use by its parity: it must not be two uses ahead of the consumers
    static_assert(RING >= NP, "each producer's blocks are NP apart");
    extern __shared__ __align__(128) unsigned char raw[];
    if (buckets) {
        behind_last_kernel();
        mark_slots(reinterpret_cast<uint32_t *>(raw + smem_bytes<K, V>(V >> (__ffs(splits) - 1))), buckets, slots_in, slots_out,
                   batch, num_slots);
    }
    Shared<K, V> &sh = *reinterpret_cast<Shared<K, V> *>(raw);
    float *buffers = reinterpret_cast<float *>(raw + sizeof(Shared<K, V>));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int split_bits = __ffs(splits) - 1, cols = V >> split_bits, consumers = cols / 16;   // splits: a power of two
    const bool whole = splits == 1;
    const long long items = (long long)batch * H * splits;
    auto bar = [&](unsigned long long &x) { return smem_u32(&x); };

    if (tid == 0) {
        for (int d = 0; d < DEPTH; ++d) {
            mbar_init(bar(sh.known[d]), 1);
            mbar_init(bar(sh.landed[d]), 1);
            mbar_init(bar(sh.done[d]), consumers);
            mbar_init(bar(sh.read[d]), NP + 1);
        }
        for (int r = 0; r < RING; ++r) {
            mbar_init(bar(sh.full[r]), 1);
            mbar_init(bar(sh.empty[r]), consumers);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    behind_last_kernel();

    // Every wait is bounded.  A warp whose wait ran out (one verdict for all its lanes) reports it and leaves without
    // another write to a state or to the ring, and without the arrival that would pass its item on: the storer finds no
    // item done that lacks a consumer, and the scout refills no buffer that was not stored.
    bool ok = false;
    auto wait = [&](unsigned long long &x, int phase) {
        return __all_sync(0xffffffffu, mbar_wait(bar(x), phase & 1, limit));
    };
    auto state_of = [&](const Item &x, int slot) {   // the item's part of a slot
        return S + (size_t)slot * slot_stride + (size_t)x.head * K * V + x.col0;
    };

    if (warp == consumers + NP) {   // scout
        const uint32_t *table = reinterpret_cast<const uint32_t *>(raw + smem_bytes<K, V>(cols));
        auto look = [&](long long at) {
            const long long chain = at >> split_bits;
            const int seq = (int)(chain / H), hi = cu[seq + 1], head = (int)(chain - (long long)seq * H);
            Item x = {cu[seq], 0, slots_in[seq], slots_out[seq], head, (int)(at & (splits - 1)) * cols};
            unsigned bad = 0;
            if (x.lo < 0 || hi < x.lo || hi > total) bad = DEV_RANGE;
            else if (x.from < -1 || x.from >= num_slots || x.to < -1 || x.to >= num_slots) bad = DEV_SLOT;
            else {
                if (x.to >= 0 && (!buckets || by_more(table, buckets, x.to)))
#pragma unroll 4
                    for (int i = lane; i < batch; i += 32)
                        if (i != seq && (slots_out[i] == x.to || slots_in[i] == x.to)) bad |= DEV_CONFLICT;
                if (index)
#pragma unroll 4
                    for (int t = x.lo + lane; t < hi; t += 32)
                        if (index[t] < 0 || index[t] >= rows) bad |= DEV_INDEX;
            }
            bad = __reduce_or_sync(0xffffffffu, bad);
            x.n = hi - x.lo;
            if (bad && lane == 0) atomicOr(status, bad);
            if (bad || (x.n == 0 && x.from == x.to)) x = {0, 0, -1, -1, 0, 0};
            return x;
        };
        int it = 0;
        for (;; ++it) {
            const long long at = blockIdx.x + (long long)it * gridDim.x;
            if ((ok = at >= items)) break;
            const int d = it % DEPTH;
            const Item x = look(at);
            // the storer is done with the buffer, the producers with the words of the item that was there
            if (!wait(sh.read[d], it / DEPTH + 1)) break;
            if (lane == 0) {
                sh.item[d] = x;
                mbar_arrive(bar(sh.known[d]));
                if (whole) {
                    mbar_arrive_expect_tx(bar(sh.landed[d]), x.from >= 0 ? (uint32_t)(4 * K * V) : 0u);
                    if (x.from >= 0)
                        bulk_g2s(smem_u32(buffers + (size_t)d * K * V), state_of(x, x.from), 4 * K * V, bar(sh.landed[d]));
                }
            }
        }
        // The block does not end before the last copies into its memory have landed, whatever the other warps' waits
        // came to: the last one of each buffer, with the usual limit.
        for (int i = max(0, it - DEPTH); whole && i < it; ++i)
            if (!mbar_wait(bar(sh.landed[i % DEPTH]), i / DEPTH & 1, WAIT_LIMIT)) ok = false;
    } else {
        int g = 0;        // token blocks so far
        int it = 0;
        for (long long at = blockIdx.x;; at += gridDim.x, ++it) {
            if ((ok = at >= items)) break;
            const int d = it % DEPTH, turn = it / DEPTH;
            if (!wait(sh.known[d], turn)) break;
            const Item x = sh.item[d];
            const int head = x.head, col0 = x.col0;
            const int blocks = (x.n + M - 1) / M;
            if (warp >= consumers && warp < consumers + NP) {   // producers
                bool free = true;
                for (int i = 0; i < blocks; ++i, ++g) {
                    if (g % NP != warp - consumers) continue;
                    if (!(free = wait(sh.empty[g % RING], g / RING + 1))) break;
                    produce<Tok, K, V>(sh.ring[g % RING], q, k, v, alpha, b, w, index, x.lo + i * M,
                                       min(M, x.n - i * M), H, head, col0, cols, lane);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(sh.full[g % RING]));
                }
                if (!free) break;
                if (lane == 0) mbar_arrive(bar(sh.read[d]));
            } else if (warp > consumers + NP) { // storer
                if (!wait(sh.done[d], turn)) break;
                if (lane == 0) {
                    if (x.to >= 0 && whole) bulk_s2g(state_of(x, x.to), smem_u32(buffers + (size_t)d * K * V), 4 * K * V);
                    bulk_commit();
                    bulk_wait_read_all();
                    mbar_arrive(bar(sh.read[d]));
                }
                __syncwarp();
            } else {                            // consumers
                float s[RJ][4][4];
                const int rg = lane >> 2, pitch = V;
                const size_t part = warp * 16 + (lane & 3) * 4 + (size_t)(4 * rg) * pitch;
                float *buffer = buffers + (size_t)d * K * V + part;
                if (whole && !wait(sh.landed[d], turn)) break;
#pragma unroll
                for (int j = 0; j < RJ; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (x.from >= 0) {
                            if (whole) y = *reinterpret_cast<const float4 *>(buffer + (32 * j + i) * pitch);
                            else y = ld_stream(reinterpret_cast<const float4 *>(state_of(x, x.from) + part + (32 * j + i) * pitch));
                        }
                        s[j][i][0] = y.x; s[j][i][1] = y.y; s[j][i][2] = y.z; s[j][i][3] = y.w;
                    }
                bool filled = true;
#pragma unroll 1
                for (int i = 0; i < blocks; ++i, ++g) {
                    // A lane's own verdict, and no branch on it: where the wait ran out the warp goes on, over whatever the
                    // ring holds, to the item's end, and leaves there (a vote for every block cost fp32 runs 5 %, this 2).
                    // It frees no slot that it did not find filled, so the other warps' blocks stay whole.
                    filled &= mbar_wait(bar(sh.full[g % RING]), g / RING & 1, filled ? limit : 0u);
                    const int t0 = x.lo + i * M, n = x.n - i * M;
                    const Block<K, V> &in = sh.ring[g % RING];
                    if (n >= 3) consume<Tok, K, V, M, OUT>(in, s, o, t0, n, H, head, col0, warp * 16, lane);
                    else if (n == 2) consume<Tok, K, V, 2, OUT>(in, s, o, t0, n, H, head, col0, warp * 16, lane);
                    else consume<Tok, K, V, 1, OUT>(in, s, o, t0, n, H, head, col0, warp * 16, lane);
                    __syncwarp();
                    if (lane == 0 && filled) mbar_arrive(bar(sh.empty[g % RING]));
                }
                if (!__all_sync(0xffffffffu, filled)) break;
                if (x.to >= 0) {
#pragma unroll
                    for (int j = 0; j < RJ; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 y = make_float4(s[j][i][0], s[j][i][1], s[j][i][2], s[j][i][3]);
                            if (whole) *reinterpret_cast<float4 *>(buffer + (32 * j + i) * pitch) = y;
                            else st_stream(reinterpret_cast<float4 *>(state_of(x, x.to) + part + (32 * j + i) * pitch), y);
                        }
                    fence_async_smem();   // the storer's bulk copy reads it
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(sh.done[d]));
            }
        }
    }
    if (!ok && lane == 0) atomicOr(status, DEV_WAIT);
}

template <typename Tok, int K, int V, bool OUT>
int launch_out(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w, float *S,
               long long slot_stride, int num_slots, const int *slots_in, const int *slots_out, const int *cu,
               const int *index, void *o, int batch, int H, int total, int rows, unsigned *status, cudaStream_t st) {
    const auto kern = recurrent_kernel<Tok, K, V, OUT>;
    constexpr size_t most = smem_bytes<K, V>(V);
    constexpr int threads = 2 * V + 32 * EXTRA_WARPS<K, V>;
    static std::atomic<int> resident{0};   // CTAs an SM; the same on every B200
    if (!allow_smem(kern, most + table_bytes(MAX_BUCKETS))) return -6;
    int per_sm = resident.load();
    if (per_sm == 0) {
        if (!succeeded(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, most)) || per_sm < 1) return -6;
        resident.store(per_sm);
    }
    // few chains: their columns over more SMs
    int splits = 1;
    while (splits < V / 16 && (long long)batch * H * splits * 2 <= 148) splits *= 2;
    const long long items = (long long)batch * H * splits, grid = items < 148 * per_sm ? items : 148 * per_sm;
    const int buckets = batch < TABLE_BATCH ? 0 : num_slots < MAX_BUCKETS ? (num_slots + 63) / 64 * 64 : MAX_BUCKETS;
    const long long polls = (long long)WAIT_LIMIT + (long long)WAIT_TOKEN * total;
    return launch_close(kern, (unsigned)grid, 2 * V / splits + 32 * EXTRA_WARPS<K, V>, smem_bytes<K, V>(V / splits) + table_bytes(buckets), st,
                        (const Tok *)q, (const Tok *)k, (const Tok *)v, alpha, (const Tok *)b, (const Tok *)w, S, slot_stride,
                        num_slots, slots_in, slots_out, cu, index, (Tok *)o, batch, H, splits, total, rows, buckets,
                        wait_limit(polls < 0xffffffffll ? (uint32_t)polls : 0xffffffffu), status);
}

template <typename Tok, int K, int V>
int launch_t(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w, float *S,
             long long slot_stride, int num_slots, const int *slots_in, const int *slots_out, const int *cu,
             const int *index, void *o, int batch, int H, int total, int rows, unsigned *status, cudaStream_t st) {
    return (o ? launch_out<Tok, K, V, true> : launch_out<Tok, K, V, false>)(q, k, v, alpha, b, w, S, slot_stride, num_slots,
                                                                         slots_in, slots_out, cu, index, o, batch, H,
                                                                         total, rows, status, st);
}

}  // namespace rec

int launch_recurrent(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w,
                     float *S, long long slot_stride, int num_slots, const int *slots_in, const int *slots_out,
                     const int *cu, const int *index, void *o, int batch, int H, int total, int rows, int K, int V,
                     int bf16, unsigned *status, cudaStream_t st) {
    auto go = [&](auto launch) {
        return launch(q, k, v, alpha, b, w, S, slot_stride, num_slots, slots_in, slots_out, cu, index, o, batch, H,
                      total, rows, status, st);
    };
    if (bf16) {
        if (K == 128) return V == 128 ? go(rec::launch_t<__nv_bfloat16, 128, 128>) : go(rec::launch_t<__nv_bfloat16, 128, 64>);
        return V == 128 ? go(rec::launch_t<__nv_bfloat16, 64, 128>) : go(rec::launch_t<__nv_bfloat16, 64, 64>);
    }
    if (K == 128) return V == 128 ? go(rec::launch_t<float, 128, 128>) : go(rec::launch_t<float, 128, 64>);
    return V == 128 ? go(rec::launch_t<float, 64, 128>) : go(rec::launch_t<float, 64, 64>);
}

}  // namespace gdn2
