// What the kernels that work on slots of a state cache share (sm_100a).
#pragma once

#include "gdn2_common.cuh"

namespace gdn2 {

// Bits of a workspace's status word for malformed device-side indices (include/gdn2.h, GDN2_DEV_*): what
// is wrong is skipped as a whole and reported, nothing is read or written out of range.
constexpr unsigned DEV_RANGE = 0x100u, DEV_SLOT = 0x200u, DEV_PARENT = 0x400u, DEV_INDEX = 0x800u,
                   DEV_CONFLICT = 0x1000u,
                   DEV_WAIT = 0x2000u;   // a bounded wait ran out

__device__ __forceinline__ float warp_sum32(float x) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// Sums of eight values over the 8 lanes of a row group (lane & 7): on return lane j holds the total of
// x[j].  Each step halves the values a lane still carries, 7 shuffles instead of 24.
__device__ __forceinline__ float scatter_sum8(const float (&x)[8], int lane) {
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

}  // namespace gdn2
