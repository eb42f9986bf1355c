// The recurrence over slots of a state cache, for ragged runs of tokens (sm_100a; page "NVIDIA представила
// Gated DeltaNet-2 ...", section "Техническая схема", the state-update equation).
//
// Sequence i owns the tokens cu[i] .. cu[i+1]-1 (through `index`, if given); its state is read from slot
// slots_in[i] and written to slot slots_out[i].  Per token, S' = Diag(alpha) S:
//   delta = w v - S'^T (b k),   S <- S' + k delta^T,   o = S^T q = S'^T q + (k.q) delta
//
// The columns of S are independent of one another, so a warp owns 16 columns from the first token to the
// last: lane = (row group rg = lane & 7, column group cg = lane >> 3), rows 4 (rg + 8 j) + i, four columns,
// which keeps the slice in K/2 registers a lane.  The two d_k-reductions are in-thread over the lane's rows
// and then over the 8 row groups by halving shuffles; no barrier stands between the tokens.  The tokens are
// staged through shared memory in fp32, STAGE at a time, in a layout in which a warp's four-row reads touch
// 128 contiguous bytes.
#include "gdn2_internal.h"
#include "gdn2_slots.cuh"

namespace gdn2 {
namespace rec {

constexpr int STAGE = 8;   // tokens staged at a time

template <int K, int V>
struct Smem {
    float a[STAGE][K], e[STAGE][K], q[STAGE][K], k[STAGE][K];   // alpha, b k, q, k
    float u[STAGE][V];                                          // w v
    float kq[STAGE];
};

// Grid: (splits, H, batch); a block owns V / splits columns of one (sequence, head), 32 threads for 16 columns.
template <typename Tok, int K, int V>
__global__ void __launch_bounds__(V * 2) recurrent_kernel(
    const Tok *__restrict__ q, const Tok *__restrict__ k, const Tok *__restrict__ v, const float *__restrict__ alpha,
    const Tok *__restrict__ b, const Tok *__restrict__ w, float *S, long long slot_stride, int num_slots,
    const int *__restrict__ slots_in, const int *__restrict__ slots_out, const int *__restrict__ cu,
    const int *__restrict__ index, Tok *__restrict__ o, int batch, int H, int total, int rows, unsigned *status) {
    constexpr int RJ = K / 32;   // groups of four rows a lane
    __shared__ __align__(16) Smem<K, V> sm;
    const int nthreads = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seq = blockIdx.z, head = blockIdx.y;
    const int col0 = (blockIdx.x * (nthreads >> 5) + warp) * 16, rg = lane & 7, cg = lane >> 3;
    const int c0 = col0 + cg * 4;

    // what the sequence asks for, checked by every block of it alike: a sequence that is malformed, or whose
    // destination another sequence names too, is left out
    const int lo = cu[seq], hi = cu[seq + 1], from = slots_in[seq], to = slots_out[seq];
    unsigned bad = 0;
    if (lo < 0 || hi < lo || hi > total) bad = DEV_RANGE;
    else if (from < -1 || from >= num_slots || to < -1 || to >= num_slots) bad = DEV_SLOT;
    else {
        if (to >= 0)
            for (int i = tid; i < batch; i += nthreads)
                if (i != seq && (slots_out[i] == to || slots_in[i] == to)) bad |= DEV_CONFLICT;
        if (index)
            for (int t = lo + tid; t < hi; t += nthreads)
                if (index[t] < 0 || index[t] >= rows) bad |= DEV_INDEX;
    }
    if (__syncthreads_or(bad != 0)) {
        if (bad) atomicOr(status, bad);
        return;
    }

    const size_t state = (size_t)head * K * V;
    float s[RJ][4][4];
#pragma unroll
    for (int j = 0; j < RJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (from >= 0)
                x = ld_stream(reinterpret_cast<const float4 *>(S + (size_t)from * slot_stride + state +
                                                               (size_t)(4 * (rg + 8 * j) + i) * V + c0));
            s[j][i][0] = x.x; s[j][i][1] = x.y; s[j][i][2] = x.z; s[j][i][3] = x.w;
        }

    for (int t0 = lo; t0 < hi; t0 += STAGE) {
        const int n = min(STAGE, hi - t0);
        __syncthreads();
        for (int i = tid; i < n * K; i += nthreads) {
            const int t = i / K, c = i % K;
            const size_t at = ((size_t)(index ? index[t0 + t] : t0 + t) * H + head) * K + c;
            const float kk = ld_tok(k + at);
            sm.a[t][c] = alpha[at];
            sm.e[t][c] = ld_tok(b + at) * kk;
            sm.q[t][c] = ld_tok(q + at);
            sm.k[t][c] = kk;
        }
        for (int i = tid; i < n * V; i += nthreads) {
            const int t = i / V, c = i % V;
            const size_t at = ((size_t)(index ? index[t0 + t] : t0 + t) * H + head) * V + c;
            sm.u[t][c] = ld_tok(w + at) * ld_tok(v + at);
        }
        __syncthreads();
        for (int t = warp; t < n; t += nthreads >> 5) {
            float d = 0.f;
#pragma unroll
            for (int c = lane; c < K; c += 32) d = fmaf(sm.k[t][c], sm.q[t][c], d);
            d = warp_sum32(d);
            if (lane == 0) sm.kq[t] = d;
        }
        __syncthreads();
        for (int t = 0; t < n; ++t) {
            float p[8];   // sums over the lane's rows: S'^T e of its four columns, S'^T q of them
#pragma unroll
            for (int c = 0; c < 8; ++c) p[c] = 0.f;
#pragma unroll
            for (int j = 0; j < RJ; ++j) {
                const float4 a4 = *reinterpret_cast<const float4 *>(&sm.a[t][4 * (rg + 8 * j)]);
                const float4 e4 = *reinterpret_cast<const float4 *>(&sm.e[t][4 * (rg + 8 * j)]);
                const float4 q4 = *reinterpret_cast<const float4 *>(&sm.q[t][4 * (rg + 8 * j)]);
                const float aa[4] = {a4.x, a4.y, a4.z, a4.w}, ee[4] = {e4.x, e4.y, e4.z, e4.w},
                            qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        s[j][i][c] *= aa[i];
                        p[c] = fmaf(ee[i], s[j][i][c], p[c]);
                        p[4 + c] = fmaf(qq[i], s[j][i][c], p[4 + c]);
                    }
            }
            const float sum = scatter_sum8(p, lane);
            // lanes rg = 0..3 hold r of column c0 + rg: delta of that column, to the whole column group
            const float mine = sm.u[t][c0 + (rg & 3)] - sum;
            float d[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) d[c] = __shfl_sync(0xffffffffu, mine, (lane & 24) | c);
            if (o && rg >= 4) {
                const float dc = rg == 4 ? d[0] : rg == 5 ? d[1] : rg == 6 ? d[2] : d[3];
                store_tok(o + ((size_t)(t0 + t) * H + head) * V + c0 + rg - 4, fmaf(sm.kq[t], dc, sum));
            }
#pragma unroll
            for (int j = 0; j < RJ; ++j) {
                const float4 k4 = *reinterpret_cast<const float4 *>(&sm.k[t][4 * (rg + 8 * j)]);
                const float kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[j][i][c] = fmaf(kk[i], d[c], s[j][i][c]);
            }
        }
    }
    if (to < 0 || (to == from && lo == hi)) return;
#pragma unroll
    for (int j = 0; j < RJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            st_stream(reinterpret_cast<float4 *>(S + (size_t)to * slot_stride + state +
                                                 (size_t)(4 * (rg + 8 * j) + i) * V + c0),
                      make_float4(s[j][i][0], s[j][i][1], s[j][i][2], s[j][i][3]));
}

template <typename Tok, int K, int V>
int launch_t(const void *q, const void *k, const void *v, const float *alpha, const void *b, const void *w, float *S,
             long long slot_stride, int num_slots, const int *slots_in, const int *slots_out, const int *cu,
             const int *index, void *o, int batch, int H, int total, int rows, unsigned *status, cudaStream_t st) {
    int splits = 1;
    while (splits < V / 16 && (long long)batch * H * splits * 2 <= 148 * 2) splits *= 2;
    recurrent_kernel<Tok, K, V><<<dim3(splits, H, batch), V * 2 / splits, 0, st>>>(
        (const Tok *)q, (const Tok *)k, (const Tok *)v, alpha, (const Tok *)b, (const Tok *)w, S, slot_stride,
        num_slots, slots_in, slots_out, cu, index, (Tok *)o, batch, H, total, rows, status);
    return launch_status();
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
