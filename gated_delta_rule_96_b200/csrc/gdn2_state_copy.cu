// Copies between slots of a state cache (sm_100a): copy, fork, compact, reorder and clear in one call.
//
// Pair i sets slot dst[i] of the destination cache to slot src[i] of the source cache (-1: zeros), as if
// every source were read before any destination is written; the two caches may be one.  A destination of
// -1 is skipped; among pairs with one destination the last one counts.
//
// Both cases move every byte once by bulk copies through shared memory.  Which one a call is, every block
// finds for itself while its first copies are on their way, from a table of the pairs' destinations:
// - No slot that changes is read: a block moves 4 KB of each of a few pairs.  4 KB pieces keep DRAM pages
//   together: compaction of 192 pairs of 1 MB takes 52 us, and 77, 67 and 60 in
//   pieces of 256, 512 and 1,024 bytes.
// - A slot that changes is read too (a reorder in place): a block owns a position range in every slot at
//   once, as much of it as shared memory holds of all pairs, and writes once all of it has landed.  No other
//   block touches the range, so any permutation needs no order among the pairs.
// The compaction runs at 5.7 TB/s of the 6.5 that a plain copy reaches; a fork (three copies of 1 MB) takes 5 us with
// cold caches and 3 behind another call.  A reorder reads its first pieces twice, and its pieces get shorter with the
// pairs: permutations of 64, 256 and 512 states of 1 MB take 27, 151 and 419 us, where twice their bytes take 21, 83 and
// 166, and one swap among 192 copies 116 us in place of 65.
#include "gdn2_internal.h"
#include "gdn2_slots.cuh"
#include "tc_ptx.cuh"

namespace gdn2 {
namespace copy {

using namespace gdn2::tc;

constexpr int THREADS = 128, RANGE = 256, GROUP = 12;   // 16-byte vectors of a piece, pairs of a block
constexpr uint32_t WAIT_LIMIT = 1u << 20;

// Shared memory: mbarrier (16 bytes), RANGE zeros, the states, the pairs, the table of destinations.
struct Layout {
    size_t pairs, total;
    int vecs, table;
};
__host__ __device__ inline Layout layout(int n, int group) {
    Layout l;
    for (l.table = 64; l.table < 2 * n; l.table *= 2) {}
    l.vecs = group * RANGE > 4 * n ? group * RANGE : 4 * n;   // 64 bytes of every pair at the least
    l.pairs = 16 + 16 * (size_t)(RANGE + l.vecs);
    l.total = l.pairs + sizeof(int) * 2 * (size_t)(n + l.table);
    return l;
}

// Grid: (position ranges of RANGE vectors, groups of `group` pairs)
__global__ void __launch_bounds__(THREADS) state_copy_kernel(float *dst, long long dst_stride, int dst_slots,
                                                             const float *src, long long src_stride, int src_slots,
                                                             const int *__restrict__ dst_idx,
                                                             const int *__restrict__ src_idx, int n, int group,
                                                             int slot_vecs, uint32_t limit, unsigned *status) {
    extern __shared__ __align__(16) unsigned char raw[];
    const Layout l = layout(n, group);
    int *s_dst = reinterpret_cast<int *>(raw + l.pairs), *s_src = s_dst + n, *s_key = s_src + n, *s_last = s_key + l.table;
    const int tid = threadIdx.x, first = blockIdx.x * RANGE, len = min(RANGE, slot_vecs - first);
    const uint32_t bar = smem_u32(raw), zeros = bar + 16, data = zeros + 16 * RANGE;

    if (tid == 0) {
        mbar_init(bar, THREADS);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < RANGE; i += THREADS) reinterpret_cast<uint4 *>(raw + 16)[i] = make_uint4(0, 0, 0, 0);
    fence_async_smem();   // the zeros are read by bulk copies
    behind_last_kernel();
    for (int i = tid; i < n; i += THREADS) {
        int d = dst_idx[i], s = src_idx[i];
        if (d < -1 || d >= dst_slots || s < -1 || s >= src_slots) {
            if (blockIdx.x == 0 && blockIdx.y == 0) atomicOr(status, DEV_SLOT);
            d = -1;
        }
        s_dst[i] = d;
        s_src[i] = s;
    }
    for (int i = tid; i < l.table; i += THREADS) s_key[i] = s_last[i] = -1;
    __syncthreads();

    // pairs lo .. hi-1, vectors at .. at+count-1 of the slots, `pitch` vectors of shared memory a pair
    auto load = [&](int lo, int hi, int at, int count, int pitch) {
        uint32_t bytes = 0;
        for (int i = lo + tid; i < hi; i += THREADS)
            if (s_dst[i] >= 0 && s_src[i] >= 0) bytes += 16 * count;
        mbar_arrive_expect_tx(bar, bytes);
        for (int i = lo + tid; i < hi; i += THREADS)
            if (s_dst[i] >= 0 && s_src[i] >= 0)
                bulk_g2s(data + 16 * (i - lo) * pitch,
                         reinterpret_cast<const uint4 *>(src + (size_t)s_src[i] * src_stride) + at, 16 * count, bar);
    };
    auto store = [&](int lo, int hi, int at, int count, int pitch) {
        for (int i = lo + tid; i < hi; i += THREADS)
            if (s_dst[i] >= 0)
                bulk_s2g(reinterpret_cast<uint4 *>(dst + (size_t)s_dst[i] * dst_stride) + at,
                         s_src[i] >= 0 ? data + 16 * (i - lo) * pitch : zeros, 16 * count);
        bulk_commit();
    };
    const int lo = blockIdx.y * group, hi = min(n, lo + group);
    load(lo, hi, first, len, RANGE);

    // the last pair of each destination: open addressing, at most half full, so every probe ends
    const auto home = [&](int d) { return (int)(((unsigned)d * 2654435761u) >> 16) & (l.table - 1); };
    for (int i = tid; i < n; i += THREADS) {
        const int d = s_dst[i];
        if (d < 0) continue;
        int at = home(d);
        for (;;) {
            const int found = atomicCAS(&s_key[at], -1, d);
            if (found == -1 || found == d) break;
            at = (at + 1) & (l.table - 1);
        }
        atomicMax(&s_last[at], i);
    }
    __syncthreads();
    const auto last = [&](int d) {   // the pair that counts for slot d, -1 if none writes it
        int at = home(d);
        while (s_key[at] != d && s_key[at] != -1) at = (at + 1) & (l.table - 1);
        return s_last[at];
    };
    bool reorder = false;
    if (dst == src)
        for (int i = tid; i < n; i += THREADS)
            if (s_dst[i] >= 0 && s_src[i] >= 0) {
                const int w = last(s_src[i]);
                reorder |= w >= 0 && s_src[w] != s_src[i];   // a slot that is written over by itself does not change
            }
    reorder = __syncthreads_or(reorder);
    // one verdict for the block, so that a round that is given up has every thread's arrival and ends all the same
    uint32_t phase = 0;
    bool ok = mbar_wait(bar, phase, limit);
    for (int i = tid; i < n; i += THREADS)
        if (s_dst[i] >= 0 && last(s_dst[i]) != i) s_dst[i] = -1;
    ok = !__syncthreads_or(!ok);
    if (!reorder) {
        if (ok) store(lo, hi, first, len, RANGE);
    } else {
        // a thread loads and stores the same pairs in every round, so its own stores are all it waits for
        const int pitch = l.vecs / n < RANGE ? l.vecs / n : RANGE;
        for (int at = blockIdx.y * pitch; ok && at < len; at += gridDim.y * pitch) {
            const int count = min(pitch, len - at);
            load(0, n, first + at, count, pitch);
            phase ^= 1;
            ok = !__syncthreads_or(!mbar_wait(bar, phase, limit));
            if (ok) store(0, n, first + at, count, pitch);
            bulk_wait_read_all();
        }
    }
    if (!ok) {   // reported and left out, after the usual wait for the round's copies, which are still on their way here
        if (tid == 0) atomicOr(status, DEV_WAIT);
        mbar_wait(bar, phase, WAIT_LIMIT);
    }
    bulk_wait_read_all();
}

}  // namespace copy

int launch_state_copy(float *dst, long long dst_stride, int dst_slots, const float *src, long long src_stride,
                      int src_slots, const int *dst_idx, const int *src_idx, int n, long long slot_floats,
                      unsigned *status, cudaStream_t st) {
    using namespace copy;
    const long long vecs = slot_floats / 4, ranges = (vecs + RANGE - 1) / RANGE;
    // up to GROUP pairs a block (four blocks share an SM), fewer while there are not two waves of such blocks
    long long group = (n * ranges + 2 * 4 * 148 - 1) / (2 * 4 * 148);
    group = group < 1 ? 1 : group > GROUP ? GROUP : group;
    const size_t smem = layout(n, (int)group).total;
    if (!allow_smem(state_copy_kernel, layout(kStateCopyMaxPairs, GROUP).total)) return -6;
    return launch_close(state_copy_kernel, dim3((unsigned)ranges, (unsigned)((n + group - 1) / group)), THREADS, smem, st, dst,
                        dst_stride, dst_slots, src, src_stride, src_slots, dst_idx, src_idx, n, (int)group, (int)vecs,
                        wait_limit(WAIT_LIMIT), status);
}

}  // namespace gdn2
