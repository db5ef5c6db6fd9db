// Row order of a batch by expert id: a stable counting sort.
//
//   order[j]   = the row at place j when the rows stand by id, rows of one id
//                in their own order, ids outside [0, E) behind all others
//   offsets[e] = rows with an id below e; expert e owns places
//                [offsets[e], offsets[e + 1])
//
// One CTA of 32 warps; warp w takes the w-th contiguous piece of the rows.
// Pass 1 counts each warp's ids in shared memory (equal ids of a warp found by
// match, one lane adds their number: no atomics, a fixed result); a scan over
// warps and ids turns counts into first places; pass 2 reads the ids again
// (L2) and writes each row to its place. Bound by latency: 8 bytes per row
// move, the largest batches take a few microseconds more than the launch.
#include "kernels.h"
#include "tiles.cuh"

namespace qlora {

namespace {

constexpr int kWarps = 32;
constexpr int kAhead = 8;  // ids of a lane in flight together

__global__ void __launch_bounds__(kWarps * 32)
    expert_order_kernel(const int* __restrict__ ids, int M, int E, int* __restrict__ order, int* __restrict__ offsets) {
    extern __shared__ int hist[];  // [kWarps][E + 1]
    __shared__ int warp_sum[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, H = E + 1;
    for (int i = threadIdx.x; i < kWarps * H; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    const int per = ((M + kWarps - 1) / kWarps + 31) & ~31;
    const int lo = min(warp * per, M), hi = min(lo + per, M);
    int* mine = hist + warp * H;
    auto key_of = [&](int row) {
        const int id = row < hi ? __ldg(ids + row) : -1;
        return id >= 0 && id < E ? id : E;
    };
    for (int b = lo; b < hi; b += 32 * kAhead) {
        int key[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) key[j] = key_of(b + 32 * j + lane);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int row = b + 32 * j + lane;
            const unsigned live = __ballot_sync(0xFFFFFFFFu, row < hi);
            if (row < hi) {
                const unsigned same = __match_any_sync(live, key[j]);
                if (lane == __ffs(same) - 1) mine[key[j]] += __popc(same);
            }
            __syncwarp();
        }
    }
    __syncthreads();
    // places of an id's rows by warp, then the ids' first places
    int total = 0;
    if (static_cast<int>(threadIdx.x) < H)
        for (int w = 0; w < kWarps; ++w) {
            const int n = hist[w * H + threadIdx.x];
            hist[w * H + threadIdx.x] = total;
            total += n;
        }
    const int incl = warp_scan_add(total);
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int s = warp_sum[lane];
        const int i = warp_scan_add(s);
        warp_sum[lane] = i - s;
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < H) {
        const int start = warp_sum[warp] + incl - total;
        offsets[threadIdx.x] = start;
        for (int w = 0; w < kWarps; ++w) hist[w * H + threadIdx.x] += start;
    }
    __syncthreads();
    for (int b = lo; b < hi; b += 32 * kAhead) {
        int key[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) key[j] = key_of(b + 32 * j + lane);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int row = b + 32 * j + lane;
            const unsigned live = __ballot_sync(0xFFFFFFFFu, row < hi);
            unsigned same = 0;
            if (row < hi) {
                same = __match_any_sync(live, key[j]);
                order[mine[key[j]] + __popc(same & ((1u << lane) - 1u))] = row;
            }
            __syncwarp();
            if (row < hi && lane == __ffs(same) - 1) mine[key[j]] += __popc(same);
            __syncwarp();
        }
    }
}

}  // namespace

cudaError_t expert_order_init_device() {
    return cudaFuncSetAttribute(expert_order_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kWarps * (kMaxExperts + 1) * 4);
}

cudaError_t launch_expert_order(const int* ids, int M, int E, int* order, int* offsets, cudaStream_t st) {
    static_assert(kMaxExperts + 1 <= kWarps * 32, "one thread per id in the scan");
    if (E < 1 || E > kMaxExperts || M < 0) return cudaErrorInvalidValue;
    expert_order_kernel<<<1, kWarps * 32, kWarps * (E + 1) * 4, st>>>(ids, M, E, order, offsets);
    return cudaGetLastError();
}

}  // namespace qlora
