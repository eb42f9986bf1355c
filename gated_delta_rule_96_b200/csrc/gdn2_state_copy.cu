// Copies between slots of a state cache (sm_100a): copy, fork, compact, reorder and clear in one call.
//
// Pair i sets slot dst[i] of the destination cache to slot src[i] of the source cache (-1: zeros), as if
// every source were read before any destination is written; the two caches may be one.  A destination of
// -1 is skipped; among pairs with one destination the last one counts.
//
// A block owns one position range of a slot, in every slot at once: it reads that range of all the pairs'
// sources into shared memory and writes them out after a barrier.  No other block touches the range, so a
// permutation in place needs no order among the pairs, and every byte is moved once.
#include "gdn2_internal.h"
#include "gdn2_slots.cuh"

namespace gdn2 {
namespace copy {

constexpr int THREADS = 256;

// Shared memory: the pairs, the table of destinations, then n * range bytes of states.
__global__ void __launch_bounds__(THREADS) state_copy_kernel(float *dst, long long dst_stride, int dst_slots,
                                                             const float *src, long long src_stride, int src_slots,
                                                             const int *__restrict__ dst_idx,
                                                             const int *__restrict__ src_idx, int n, int range,
                                                             int slot_vecs, unsigned *status) {
    extern __shared__ __align__(16) unsigned char raw[];
    int *s_dst = reinterpret_cast<int *>(raw), *s_src = s_dst + n;
    const int tid = threadIdx.x;
    int table = 1;
    while (table < 2 * n) table *= 2;
    int *s_key = s_src + n, *s_last = s_key + table;
    uint4 *s_data = reinterpret_cast<uint4 *>(raw + ((2 * (size_t)(n + table) * sizeof(int) + 15) & ~(size_t)15));

    for (int i = tid; i < table; i += THREADS) s_key[i] = -1, s_last[i] = -1;
    for (int i = tid; i < n; i += THREADS) {
        int d = dst_idx[i], s = src_idx[i];
        if (d < -1 || d >= dst_slots || s < -1 || s >= src_slots) {
            if (blockIdx.x == 0) atomicOr(status, DEV_SLOT);
            d = -1;
        }
        s_dst[i] = d;
        s_src[i] = s;
    }
    __syncthreads();
    // the last pair of each destination: open addressing, at most half full, so every probe ends
    for (int i = tid; i < n; i += THREADS) {
        const int d = s_dst[i];
        if (d < 0) continue;
        int at = (int)(((unsigned)d * 2654435761u) >> 16) & (table - 1);
        for (;;) {
            const int found = atomicCAS(&s_key[at], -1, d);
            if (found == -1 || found == d) break;
            at = (at + 1) & (table - 1);
        }
        atomicMax(&s_last[at], i);
    }
    __syncthreads();
    for (int i = tid; i < n; i += THREADS) {
        const int d = s_dst[i];
        if (d < 0) continue;
        int at = (int)(((unsigned)d * 2654435761u) >> 16) & (table - 1);
        while (s_key[at] != d) at = (at + 1) & (table - 1);
        if (s_last[at] != i) s_dst[i] = -1;
    }
    __syncthreads();

    const int first = blockIdx.x * range, len = min(range, slot_vecs - first), vecs = n * range;
    for (int i = tid; i < vecs; i += THREADS) {
        const int p = i / range, c = i - p * range;
        if (s_dst[p] < 0 || c >= len) continue;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (s_src[p] >= 0)
            x = __ldcs(reinterpret_cast<const uint4 *>(src + (size_t)s_src[p] * src_stride) + first + c);
        s_data[i] = x;
    }
    __syncthreads();
    for (int i = tid; i < vecs; i += THREADS) {
        const int p = i / range, c = i - p * range;
        if (s_dst[p] < 0 || c >= len) continue;
        __stcs(reinterpret_cast<uint4 *>(dst + (size_t)s_dst[p] * dst_stride) + first + c, s_data[i]);
    }
}

}  // namespace copy

int launch_state_copy(float *dst, long long dst_stride, int dst_slots, const float *src, long long src_stride,
                      int src_slots, const int *dst_idx, const int *src_idx, int n, long long slot_floats,
                      unsigned *status, cudaStream_t st) {
    int table = 1;
    while (table < 2 * n) table *= 2;
    const size_t head = (2 * (size_t)(n + table) * sizeof(int) + 15) & ~(size_t)15;
    // the range of a block, in 16-byte vectors: up to 4 KB, as large as lets two blocks share an SM
    int range = 256;
    while (range > 8 && head + (size_t)n * range * 16 > 100 * 1024) range /= 2;
    const size_t smem = head + (size_t)n * range * 16;
    const long long vecs = slot_floats / 4, blocks = (vecs + range - 1) / range;
    if (cudaFuncSetAttribute(copy::state_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess)
        return -6;
    copy::state_copy_kernel<<<(unsigned)blocks, copy::THREADS, smem, st>>>(dst, dst_stride, dst_slots, src, src_stride,
                                                                          src_slots, dst_idx, src_idx, n, range,
                                                                          (int)vecs, status);
    return launch_status();
}

}  // namespace gdn2
