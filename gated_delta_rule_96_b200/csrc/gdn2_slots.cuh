// What the kernels that work on slots of a state cache share (sm_100a).
#pragma once

#include "gdn2_common.cuh"

namespace gdn2 {

// Bits of a workspace's status word for malformed device-side indices (include/gdn2.h, GDN2_DEV_*): what
// is wrong is skipped as a whole and reported, nothing is read or written out of range.
constexpr unsigned DEV_RANGE = 0x100u, DEV_SLOT = 0x200u, DEV_PARENT = 0x400u, DEV_INDEX = 0x800u,
                   DEV_CONFLICT = 0x1000u,
                   DEV_WAIT = 0x2000u;   // a bounded wait ran out

// N consecutive token elements, as they are stored and as fp32
template <typename Tok, int N>
struct Raw {
    static constexpr int W = N * (int)sizeof(Tok) / 4;
    uint32_t r[W];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < W; ++i) r[i] = 0u;
    }
    __device__ __forceinline__ void load(const Tok *p) {   // N * sizeof(Tok) <= 16 bytes, aligned to them
        if constexpr (W == 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
        } else if constexpr (W == 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            r[0] = v.x; r[1] = v.y;
        } else {
            r[0] = *reinterpret_cast<const uint32_t *>(p);
        }
    }
    __device__ __forceinline__ void get(float (&x)[N]) const {
        if constexpr (sizeof(Tok) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = __uint_as_float(r[i]);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) {   // bf16 is the upper half of an fp32
                x[2 * i] = __uint_as_float(r[i] << 16);
                x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
            }
        }
    }
};

// Two fp32 in one register pair: half the issue slots of the scalar form at the same rate of the FMA pipe
// (measured 71 against 67 TFLOP/s), for kernels that the issue slots bound.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// four consecutive floats as two pairs
__device__ __forceinline__ void load2(const float *p, f32x2 (&x)[2]) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
    x[0] = v.x;
    x[1] = v.y;
}

// Sums of eight values over the 8 row groups (lane >> 2, the column groups on the low bits): on return row
// group j holds the total of x[j].  Each step halves the values a lane still carries, 7 shuffles instead of 24.
__device__ __forceinline__ float scatter_sum8(const float (&x)[8], int lane) {
    float a[4], b[2];
    const bool up4 = lane & 16, up2 = lane & 8, up1 = lane & 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a[i] = (up4 ? x[i + 4] : x[i]) + __shfl_xor_sync(0xffffffffu, up4 ? x[i] : x[i + 4], 16);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        b[i] = (up2 ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, up2 ? a[i] : a[i + 2], 8);
    return (up1 ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, up1 ? b[0] : b[1], 4);
}

}  // namespace gdn2
