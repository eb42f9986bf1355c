// The layer's norms (sm_100a): the gated RMSNorm behind the mixer and the residual RMSNorm before the
// next block, each with its gradients.
//
// Gated norm, per row of d_v channels:   x^ = o r,  r = (mean(o^2) + eps)^(-1/2),  y = x^ weight act(g)
//   backward, dn = dy act(g):  dg = dy x^ weight act'(g),  dx^ = dn weight,
//                              do = r (dx^ - x^ mean(dx^ x^)),  dweight = sum_rows dn x^
// Residual norm, per row of `width` channels:   h = residual + scale x,  y = h r(h) weight
//   backward, at the stored h:  dresidual = dh + r (dy weight - h^ mean(dy weight h^)),
//                               dx = scale dresidual,  dscale = sum_rows dresidual x,  dweight = sum_rows dy h^
// Both are one pass over their tensors: a row lives in the registers of the threads that own it, the
// row sums are fp32 shuffles (and one exchange through shared memory where a row spans warps), and every
// output is rounded once.  The column sums are fp32 per thread over the rows that it walks, then added in
// a fixed order (per block, then over the blocks by a second kernel), so results do not change from run
// to run.  HBM bounds them all.  One call behind another, gated norm of 524,288 rows of 128 bf16: forward 64 us (6.3 TB/s of the
// 6.5 that a copy reaches), backward 113 us (5.9).  A single launch's device time is shorter, 61 and 109 us, since its last
// writes are still in L2 when it ends; so measured the residual norm of 32,768 rows of 2,048 takes 79 us forward and 139
// backward, the sum over the blocks 5-7 us, and a few rows (a decode step) 3-4 us, latency alone.
#include "gdn2_common.cuh"
#include "gdn2_internal.h"

namespace gdn2 {
namespace norms {

// 16 bytes of tokens as fp32
template <typename Tok>
struct V16;
template <>
struct V16<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[8]) {
        const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // bf16 is the upper half of an fp32
            x[2 * i] = __uint_as_float(p[i] << 16);
            x[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            p[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(p[0], p[1], p[2], p[3]);
    }
};
template <>
struct V16<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

// N consecutive fp32 weights (N = 4 or 8, 16-byte aligned)
template <int N>
__device__ __forceinline__ void load_f32(const float *p, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p + i);
        x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    }
}

// sum over groups of LANES consecutive lanes
template <int LANES>
__device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

struct Sigmoid {
    float s, c;   // sigmoid(x), and one less it without the cancellation that the difference has above zero
};
template <typename Tok>
__device__ __forceinline__ Sigmoid sigmoid_(float x) {
    if constexpr (sizeof(Tok) == 4) {
        // fp32 tokens keep fp32's precision, within a few units whatever x is; twice the bytes hide most of it (524,288
        // rows of 128, with the form below / with this: forward 118 / 118 us, backward 224 / 234; of 64 110 / 106)
        const float e = expf(-fabsf(x)), r = 1.f / (1.f + e), p = e * r;
        return x >= 0.f ? Sigmoid{r, p} : Sigmoid{p, r};
    } else {
        // 1 / (1 + 2^(-x log2 e)) on the special-function unit: two instructions there and two beside them, where
        // expf and the divide take some twenty, which bounded the kernels at two thirds of the copy rate.  Each of
        // the two is good to about one unit of fp32 and the argument's rounding adds |x| / 2 more, where the output's
        // rounding to bf16 is up to 2^16 units; the ends are exact.
        float e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
        return {r, x > 0.f ? e * r : 1.f - r};
    }
}

constexpr int ACT_SILU = 0;

// ---------------------------------------------------------------- gated norm

// A row of D channels is held by LPR lanes, 16 bytes each; a thread has U rows in flight.
template <typename Tok, int D, int ACT, int U>
__global__ void __launch_bounds__(256) gated_norm_fwd_kernel(const Tok *o, const Tok *gate,
                                                             const float *__restrict__ weight, Tok *y,
                                                             long long rows, float eps) {
    behind_last_kernel();
    using V = V16<Tok>;
    constexpr int N = V::N, LPR = D / N, RPW = 32 / LPR;
    const int lane = threadIdx.x & 31, sub = lane % LPR;
    const long long first = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * (RPW * U) + lane / LPR;
    float wt[N];
    load_f32<N>(weight + sub * N, wt);
    uint4 xo[U], xg[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long r = first + u * RPW;
        xo[u] = xg[u] = make_uint4(0, 0, 0, 0);
        if (r < rows) {
            xo[u] = __ldcs(reinterpret_cast<const uint4 *>(o + r * D) + sub);
            xg[u] = __ldcs(reinterpret_cast<const uint4 *>(gate + r * D) + sub);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long r = first + u * RPW;
        float x[N], g[N], ss = 0.f;
        V::unpack(xo[u], x);
        V::unpack(xg[u], g);
#pragma unroll
        for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
        const float inv = rsqrtf(lane_sum<LPR>(ss) * (1.f / D) + eps);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float s = sigmoid_<Tok>(g[i]).s;
            x[i] = x[i] * inv * wt[i] * (ACT == ACT_SILU ? g[i] * s : s);
        }
        if (r < rows) __stcs(reinterpret_cast<uint4 *>(y + r * D) + sub, V::pack(x));
    }
}

template <typename Tok, int D, int ACT>
__global__ void __launch_bounds__(256) gated_norm_bwd_kernel(const Tok *__restrict__ o, const Tok *__restrict__ gate,
                                                             const float *__restrict__ weight,
                                                             const Tok *__restrict__ dy, Tok *__restrict__ d_o,
                                                             Tok *__restrict__ dgate, float *__restrict__ partial,
                                                             long long rows, float eps) {
    behind_last_kernel();
    using V = V16<Tok>;
    constexpr int N = V::N, LPR = D / N, RPW = 32 / LPR;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPR;
    float wt[N], dw[N];
    load_f32<N>(weight + sub * N, wt);
#pragma unroll
    for (int i = 0; i < N; ++i) dw[i] = 0.f;
    const long long step = (long long)gridDim.x * 8 * RPW;
    uint4 xo, xg, xy;   // the next rows are on their way while these are worked on
    auto fetch = [&](long long r) {
        xo = xg = xy = make_uint4(0, 0, 0, 0);
        if (r < rows) {
            xo = __ldcs(reinterpret_cast<const uint4 *>(o + r * D) + sub);
            xg = __ldcs(reinterpret_cast<const uint4 *>(gate + r * D) + sub);
            xy = __ldcs(reinterpret_cast<const uint4 *>(dy + r * D) + sub);
        }
    };
    // rows are walked by whole warps: the shuffles below need every lane
    long long r0 = ((long long)blockIdx.x * 8 + warp) * RPW;
    fetch(r0 + lane / LPR);
    for (; r0 < rows; r0 += step) {
        const long long r = r0 + lane / LPR;
        float x[N], g[N], d[N], ss = 0.f, sd = 0.f;
        V::unpack(xo, x);
        V::unpack(xg, g);
        V::unpack(xy, d);
        fetch(r + step);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const auto [s, c] = sigmoid_<Tok>(g[i]);
            const float act = ACT == ACT_SILU ? g[i] * s : s;
            const float slope = ACT == ACT_SILU ? s * (1.f + g[i] * (1.f - s)) : s * c;
            ss = fmaf(x[i], x[i], ss);
            const float dn = d[i] * act;                  // d(x^ weight)
            sd = fmaf(dn * wt[i], x[i], sd);
            g[i] = d[i] * x[i] * wt[i] * slope;           // dgate / r
            d[i] = dn;
        }
        ss = lane_sum<LPR>(ss);
        sd = lane_sum<LPR>(sd);
        const float inv = r < rows ? rsqrtf(ss * (1.f / D) + eps) : 0.f;   // eps may be 0
        const float mean = sd * inv * inv * (1.f / D);    // mean(dx^ x^) r, to be multiplied by o
        float out[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            dw[i] = fmaf(d[i], x[i] * inv, dw[i]);
            out[i] = inv * (d[i] * wt[i] - x[i] * mean);
            g[i] *= inv;
        }
        if (r < rows) {
            __stcs(reinterpret_cast<uint4 *>(d_o + r * D) + sub, V::pack(out));
            __stcs(reinterpret_cast<uint4 *>(dgate + r * D) + sub, V::pack(g));
        }
    }
    __shared__ float s_dw[8][D];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float t = dw[i];
#pragma unroll
        for (int m = LPR; m < 32; m <<= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
        if (lane < LPR) s_dw[warp][sub * N + i] = t;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += 256) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += s_dw[w][c];
        partial[(size_t)blockIdx.x * D + c] = t;
    }
}

// out[c] = sum over g of partial[g][c], in a fixed order: 32 columns a block, 32 row groups
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *__restrict__ partial, int groups, int columns,
                                                          float *__restrict__ out0, float *__restrict__ out1,
                                                          int split) {
    behind_last_kernel();
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < columns)
        for (int g = part; g < groups; g += 32) t += partial[(size_t)g * columns + c];
    s[part][lane] = t;
    __syncthreads();
    t = lane_sum<32>(s[lane][part]);
    if (lane == 0) {
        const int col = blockIdx.x * 32 + part;
        if (col < split) out0[col] = t;
        else if (col < columns) out1[col - split] = t;
    }
}

// ---------------------------------------------------------------- residual norm

// A row is eight lanes' to sixteen warps', and a block has eight warps or one row.  Forward the row's loads are in flight at once,
// and 2,048 threads an SM hide them.  Backward a block walks rows, since it carries the columns' sums: two blocks an SM; loading the next row ahead took 151 us where this
// takes 143, two vectors a thread 145.

// Sum over the `warps` warps of a row, `first` of them the first, of up to two values at once; `s` is one of two buffers
// taken in turn, so that one barrier a row is enough.  The whole block calls it.  LANES below 32: a row is as many
// lanes of a warp.
template <int C, int LANES>
__device__ __forceinline__ void row_sum(float (&x)[C], float (*s)[C], int first, int warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = lane_sum<LANES>(x[c]);
    if (LANES < 32 || warps == 1) return;
    if (lane == 0)
#pragma unroll
        for (int c = 0; c < C; ++c) s[warp][c] = x[c];
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c) {
        x[c] = 0.f;
        for (int w = 0; w < warps; ++w) x[c] += s[first + w][c];
    }
}

constexpr int MAX_WARPS = 16;   // of a block: rows of up to 512 threads
constexpr int MAX_WIDTH = 8192;

template <typename Tok, int NV, int SHARE>
__global__ void __launch_bounds__(512) add_norm_fwd_kernel(const Tok *x, const Tok *residual,
                                                           const float *__restrict__ scale,
                                                           const float *__restrict__ weight, Tok *h, Tok *y,
                                                           long long rows, int vecs, int row_warps, float eps) {
    behind_last_kernel();
    // the block's rows, and the thread's place in its own
    const int row_threads = SHARE == 0 ? blockDim.x : SHARE == 32 ? 32 * row_warps : SHARE,
              team = SHARE == 0 ? 0 : SHARE == 32 ? (threadIdx.x >> 5) / row_warps : threadIdx.x / SHARE,
              teams = SHARE == 0 ? 1 : SHARE == 32 ? (blockDim.x >> 5) / row_warps : blockDim.x / SHARE,
              at = threadIdx.x - team * row_threads;
    using V = V16<Tok>;
    constexpr int N = V::N;
    __shared__ float s_sum[2][MAX_WARPS][1];
    const float inv_width = 1.f / (float)(vecs * N);
    int flip = 0;
    for (long long r0 = (long long)blockIdx.x * teams; r0 < rows; r0 += (long long)gridDim.x * teams, flip ^= 1) {
        const size_t base = (size_t)(r0 + team) * vecs;
        const int mine = !SHARE || r0 + team < rows ? vecs : 0;
        uint4 xr[NV], rr[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = at + j * row_threads;
            xr[j] = rr[j] = make_uint4(0, 0, 0, 0);
            if (v < mine) {
                xr[j] = __ldcs(reinterpret_cast<const uint4 *>(x) + base + v);
                if (residual) rr[j] = __ldcs(reinterpret_cast<const uint4 *>(residual) + base + v);
            }
        }
        float a[NV][N], sum[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = at + j * row_threads;
            float xf[N], sc[N];
            V::unpack(xr[j], xf);
            V::unpack(rr[j], a[j]);
            if (scale && v < mine) load_f32<N>(scale + (size_t)v * N, sc);
            else
#pragma unroll
                for (int i = 0; i < N; ++i) sc[i] = 1.f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                a[j][i] = fmaf(sc[i], xf[i], a[j][i]);
                sum[0] = fmaf(a[j][i], a[j][i], sum[0]);
            }
            if (h && v < mine) __stcs(reinterpret_cast<uint4 *>(h) + base + v, V::pack(a[j]));
        }
        row_sum<1, SHARE == 0 ? 32 : SHARE>(sum, s_sum[flip], team * row_warps, SHARE ? row_warps : blockDim.x >> 5);
        const float inv = rsqrtf(sum[0] * inv_width + eps);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = at + j * row_threads;
            if (v < mine) {
                float wt[N];
                load_f32<N>(weight + (size_t)v * N, wt);
#pragma unroll
                for (int i = 0; i < N; ++i) a[j][i] *= inv * wt[i];
                __stcs(reinterpret_cast<uint4 *>(y) + base + v, V::pack(a[j]));
            }
        }
    }
}

template <typename Tok, int NV, bool SCALED, int SHARE>
__global__ void __launch_bounds__(512, NV == 1 ? 2 : 1) add_norm_bwd_kernel(const Tok *__restrict__ h, const Tok *__restrict__ x,
                                                           const float *__restrict__ scale,
                                                           const float *__restrict__ weight,
                                                           const Tok *__restrict__ dy, const Tok *__restrict__ dh,
                                                           Tok *__restrict__ dres, Tok *__restrict__ dx,
                                                           float *__restrict__ partial, long long rows, int vecs,
                                                           int row_warps, float eps) {
    behind_last_kernel();
    // the block's rows, and the thread's place in its own
    const int row_threads = SHARE == 0 ? blockDim.x : SHARE == 32 ? 32 * row_warps : SHARE,
              team = SHARE == 0 ? 0 : SHARE == 32 ? (threadIdx.x >> 5) / row_warps : threadIdx.x / SHARE,
              teams = SHARE == 0 ? 1 : SHARE == 32 ? (blockDim.x >> 5) / row_warps : blockDim.x / SHARE,
              at = threadIdx.x - team * row_threads;
    using V = V16<Tok>;
    constexpr int N = V::N;
    __shared__ float s_sum[2][MAX_WARPS][2];
    const int width = vecs * N;
    const float inv_width = 1.f / (float)width;
    extern __shared__ __align__(16) float s_weights[];   // weight, then scale: registers go to rows in flight
    float dw[NV][N], ds[NV][N];
    for (int c = 4 * threadIdx.x; c < width; c += 4 * blockDim.x) {
        *reinterpret_cast<float4 *>(s_weights + c) = *reinterpret_cast<const float4 *>(weight + c);
        if (SCALED) *reinterpret_cast<float4 *>(s_weights + width + c) = *reinterpret_cast<const float4 *>(scale + c);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) dw[j][i] = ds[j][i] = 0.f;
    __syncthreads();
    int flip = 0;
    for (long long r0 = (long long)blockIdx.x * teams; r0 < rows; r0 += (long long)gridDim.x * teams, flip ^= 1) {
        const size_t base = (size_t)(r0 + team) * vecs;
        const bool live = !SHARE || r0 + team < rows;
        uint4 hr[NV], xr[NV], yr[NV], gr[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = at + j * row_threads;
            hr[j] = xr[j] = yr[j] = gr[j] = make_uint4(0, 0, 0, 0);
            if (live && v < vecs) {
                hr[j] = __ldcs(reinterpret_cast<const uint4 *>(h) + base + v);
                yr[j] = __ldcs(reinterpret_cast<const uint4 *>(dy) + base + v);
                if (SCALED) xr[j] = __ldcs(reinterpret_cast<const uint4 *>(x) + base + v);
                if (dh) gr[j] = __ldcs(reinterpret_cast<const uint4 *>(dh) + base + v);
            }
        }
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = at + j * row_threads;
            float hf[N], df[N], wt[N];
            V::unpack(hr[j], hf);
            V::unpack(yr[j], df);
            load_f32<N>(s_weights + (v < vecs ? v : 0) * N, wt);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                sum[0] = fmaf(hf[i], hf[i], sum[0]);
                sum[1] = fmaf(df[i] * wt[i], hf[i], sum[1]);
            }
        }
        row_sum<2, SHARE == 0 ? 32 : SHARE>(sum, s_sum[flip], team * row_warps, SHARE ? row_warps : blockDim.x >> 5);
        const float inv = live ? rsqrtf(sum[0] * inv_width + eps) : 0.f;   // eps may be 0
        const float mean = sum[1] * inv * inv * inv_width;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = at + j * row_threads;
            float hf[N], df[N], gf[N], wt[N];
            V::unpack(hr[j], hf);
            V::unpack(yr[j], df);
            V::unpack(gr[j], gf);
            load_f32<N>(s_weights + (v < vecs ? v : 0) * N, wt);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                dw[j][i] = fmaf(df[i], hf[i] * inv, dw[j][i]);
                gf[i] += inv * (df[i] * wt[i] - hf[i] * mean);
            }
            if (live && v < vecs) __stcs(reinterpret_cast<uint4 *>(dres) + base + v, V::pack(gf));
            if (SCALED) {
                float xf[N], sc[N];
                V::unpack(xr[j], xf);
                load_f32<N>(s_weights + width + (v < vecs ? v : 0) * N, sc);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    ds[j][i] = fmaf(gf[i], xf[i], ds[j][i]);
                    gf[i] *= sc[i];
                }
                if (live && v < vecs) __stcs(reinterpret_cast<uint4 *>(dx) + base + v, V::pack(gf));
            }
        }
    }
    // the block's rows added up, one after the other, in place of the weights
    for (int t = 0; SHARE && t < teams; ++t) {
        __syncthreads();
        if (team != t) continue;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = at + j * row_threads;
            if (v >= vecs) continue;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float *w = s_weights + v * N + i;
                *w = dw[j][i] += t ? *w : 0.f;
                if (SCALED) w[width] = ds[j][i] += t ? w[width] : 0.f;
            }
        }
    }
    if (team != teams - 1) return;
    float *mine = partial + (size_t)blockIdx.x * width * (SCALED ? 2 : 1);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = at + j * row_threads;
        if (v < vecs)
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                *reinterpret_cast<float4 *>(mine + (size_t)v * N + i) =
                    make_float4(dw[j][i], dw[j][i + 1], dw[j][i + 2], dw[j][i + 3]);
                if (SCALED)
                    *reinterpret_cast<float4 *>(mine + width + (size_t)v * N + i) =
                        make_float4(ds[j][i], ds[j][i + 1], ds[j][i + 2], ds[j][i + 3]);
            }
    }
}

// The backward kernels' blocks walk the rows, each with one row of partial column sums at its end: as many
// as are resident at once (a second, partial wave of such blocks costs as much as the first), at most
// MAX_BLOCKS.
constexpr int SMS = 148, MAX_BLOCKS = 4 * SMS;
int cap_blocks(long long want, int per_sm) {
    const long long most = per_sm < 4 ? (per_sm < 1 ? 1 : per_sm) * SMS : MAX_BLOCKS;
    return (int)(want < most ? (want > 0 ? want : 1) : most);
}
template <typename Kernel>
int resident(Kernel kern, int threads, size_t smem) {
    int n = 0;
    return succeeded(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem)) ? n : 1;
}

// warps that hold a row of `vecs` 16-byte vectors, NV a thread, and the rows of a block: narrow rows share one, since
// blocks of a warp leave most of an SM empty (forward and backward, us, a row and several rows a block: 149,421 rows of
// 208 bf16 306 / 98, 60,000 of 512 bf16 182 / 114, 32,768 of 1,024 bf16 138 / 122), and up to 16 vectors a warp, since
// lanes without a vector do too (a row and several rows a warp: 400,000 of 64 bf16 234 / 94, 250,000 of 128 155 / 108)
int row_warps(int vecs, int nv) { return ((vecs + nv - 1) / nv + 31) / 32; }
int block_rows(int vecs, int warps) { return vecs <= 8 ? 32 : vecs <= 16 ? 16 : warps < 8 ? 8 / warps : 1; }

template <typename Tok, int D, int ACT>
int gated_fwd_t(const void *o, const void *gate, const float *weight, void *y, long long rows, float eps,
                cudaStream_t st) {
    constexpr int PER_BLOCK = 8 * 32 / (D / V16<Tok>::N);
    // four rows a thread in flight hide the latency of a long stream; a few rows are spread over more blocks
    auto go = [&](auto kern, int u) {
        const long long per_block = (long long)PER_BLOCK * u;
        return launch_close(kern, (unsigned)((rows + per_block - 1) / per_block), 256, 0, st, (const Tok *)o, (const Tok *)gate,
                            weight, (Tok *)y, rows, eps);
    };
    return rows >= (long long)PER_BLOCK * 4 * SMS * 2 ? go(gated_norm_fwd_kernel<Tok, D, ACT, 4>, 4)
                                                      : go(gated_norm_fwd_kernel<Tok, D, ACT, 1>, 1);
}
template <typename Tok, int D, int ACT>
int gated_bwd_t(const void *o, const void *gate, const float *weight, const void *dy, void *d_o, void *dgate,
                float *dweight, long long rows, float eps, float *partial, cudaStream_t st) {
    static const int per_sm = resident(gated_norm_bwd_kernel<Tok, D, ACT>, 256, 0);   // the same on every B200
    const int blocks = cap_blocks((rows + 7) / 8, per_sm);
    const int rc = launch_close(gated_norm_bwd_kernel<Tok, D, ACT>, blocks, 256, 0, st, (const Tok *)o, (const Tok *)gate, weight,
                                (const Tok *)dy, (Tok *)d_o, (Tok *)dgate, partial, rows, eps);
    return rc ? rc : launch_close(column_sum_kernel, D / 32, 1024, 0, st, partial, blocks, D, dweight, nullptr, D);
}

template <typename Tok>
int add_fwd_t(const void *x, const void *residual, const float *scale, const float *weight, void *h, void *y,
              long long rows, int width, float eps, cudaStream_t st) {
    const int vecs = width / V16<Tok>::N, nv = vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4, warps = row_warps(vecs, nv), teams = block_rows(vecs, warps), nt = teams > 8 ? 256 : 32 * warps * teams;
    const long long want = (rows + teams - 1) / teams;
    const unsigned blocks = (unsigned)(want < (1 << 30) ? want : (1 << 30));
    auto go = [&](auto kern) {
        return launch_close(kern, blocks, nt, 0, st, (const Tok *)x, (const Tok *)residual, scale, weight, (Tok *)h, (Tok *)y, rows,
                            vecs, warps, eps);
    };
    if (teams == 32) return go(add_norm_fwd_kernel<Tok, 1, 8>);
    if (teams == 16) return go(add_norm_fwd_kernel<Tok, 1, 16>);
    if (teams > 1) return go(add_norm_fwd_kernel<Tok, 1, 32>);
    if (nv == 1) return go(add_norm_fwd_kernel<Tok, 1, 0>);
    if (nv == 2) return go(add_norm_fwd_kernel<Tok, 2, 0>);
    if constexpr (sizeof(Tok) == 4) return go(add_norm_fwd_kernel<Tok, 4, 0>);
    return -6;   // bf16 rows end at 1024 vectors
}
template <typename Tok, bool SCALED>
int add_bwd_t(const void *h, const void *x, const float *scale, const float *weight, const void *dy, const void *dh,
              void *dres, void *dx, float *dscale, float *dweight, long long rows, int width, float eps,
              float *partial, cudaStream_t st) {
    const int vecs = width / V16<Tok>::N, nv = vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4, warps = row_warps(vecs, nv), teams = block_rows(vecs, warps), nt = teams > 8 ? 256 : 32 * warps * teams;
    const int columns = width * (SCALED ? 2 : 1);
    int blocks = 0;
    int rc = -6;
    auto go = [&](auto kern) {
        const size_t smem = sizeof(float) * (size_t)columns;
        if (!allow_smem(kern, sizeof(float) * 2 * MAX_WIDTH)) return;
        blocks = cap_blocks((rows + teams - 1) / teams, resident(kern, nt, smem));
        rc = launch_close(kern, blocks, nt, smem, st, (const Tok *)h, (const Tok *)x, scale, weight, (const Tok *)dy, (const Tok *)dh,
                          (Tok *)dres, (Tok *)dx, partial, rows, vecs, warps, eps);
    };
    if (teams == 32) go(add_norm_bwd_kernel<Tok, 1, SCALED, 8>);
    else if (teams == 16) go(add_norm_bwd_kernel<Tok, 1, SCALED, 16>);
    else if (teams > 1) go(add_norm_bwd_kernel<Tok, 1, SCALED, 32>);
    else if (nv == 1) go(add_norm_bwd_kernel<Tok, 1, SCALED, 0>);
    else if (nv == 2) go(add_norm_bwd_kernel<Tok, 2, SCALED, 0>);
    else if constexpr (sizeof(Tok) == 4) go(add_norm_bwd_kernel<Tok, 4, SCALED, 0>);   // bf16 rows end at 1024 vectors
    return rc ? rc : launch_close(column_sum_kernel, (columns + 31) / 32, 1024, 0, st, partial, blocks, columns, dweight, dscale, width);
}

}  // namespace norms

size_t gated_norm_bwd_workspace_bytes(long long rows, int D) {
    return kStatusBytes + sizeof(float) * (size_t)norms::cap_blocks((rows + 7) / 8, 4) * D;
}
size_t add_norm_bwd_workspace_bytes(long long rows, int width) {
    return kStatusBytes + sizeof(float) * (size_t)norms::cap_blocks(rows, 4) * width * 2;
}

int launch_gated_norm_fwd(const void *o, const void *gate, const float *weight, void *y, long long rows, int D, int act,
                          float eps, int bf16, cudaStream_t st) {
    using namespace norms;
    using bf = __nv_bfloat16;
#define GDN2_GATED(T, DD, A) return gated_fwd_t<T, DD, A>(o, gate, weight, y, rows, eps, st)
#define GDN2_GATED_ACT(T, DD) do { if (act == 0) GDN2_GATED(T, DD, 0); GDN2_GATED(T, DD, 1); } while (0)
    if (bf16) {
        if (D == 128) GDN2_GATED_ACT(bf, 128);
        GDN2_GATED_ACT(bf, 64);
    }
    if (D == 128) GDN2_GATED_ACT(float, 128);
    GDN2_GATED_ACT(float, 64);
#undef GDN2_GATED
}

int launch_gated_norm_bwd(const void *o, const void *gate, const float *weight, const void *dy, void *d_o, void *dgate,
                          float *dweight, long long rows, int D, int act, float eps, int bf16, void *ws,
                          cudaStream_t st) {
    using namespace norms;
    using bf = __nv_bfloat16;
    float *partial = reinterpret_cast<float *>(static_cast<char *>(ws) + kStatusBytes);
#define GDN2_GATED(T, DD, A) return gated_bwd_t<T, DD, A>(o, gate, weight, dy, d_o, dgate, dweight, rows, eps, partial, st)
    if (bf16) {
        if (D == 128) GDN2_GATED_ACT(bf, 128);
        GDN2_GATED_ACT(bf, 64);
    }
    if (D == 128) GDN2_GATED_ACT(float, 128);
    GDN2_GATED_ACT(float, 64);
#undef GDN2_GATED
#undef GDN2_GATED_ACT
}

int launch_add_norm_fwd(const void *x, const void *residual, const float *scale, const float *weight, void *h, void *y,
                        long long rows, int width, float eps, int bf16, cudaStream_t st) {
    if (bf16) return norms::add_fwd_t<__nv_bfloat16>(x, residual, scale, weight, h, y, rows, width, eps, st);
    return norms::add_fwd_t<float>(x, residual, scale, weight, h, y, rows, width, eps, st);
}

int launch_add_norm_bwd(const void *h, const void *x, const float *scale, const float *weight, const void *dy,
                        const void *dh, void *dres, void *dx, float *dscale, float *dweight, long long rows, int width,
                        float eps, int bf16, void *ws, cudaStream_t st) {
    using namespace norms;
    using bf = __nv_bfloat16;
    float *partial = reinterpret_cast<float *>(static_cast<char *>(ws) + kStatusBytes);
#define GDN2_ADD(T, S) return add_bwd_t<T, S>(h, x, scale, weight, dy, dh, dres, dx, dscale, dweight, rows, width, eps, partial, st)
    if (bf16) {
        if (scale) GDN2_ADD(bf, true);
        GDN2_ADD(bf, false);
    }
    if (scale) GDN2_ADD(float, true);
    GDN2_ADD(float, false);
#undef GDN2_ADD
}

}  // namespace gdn2
