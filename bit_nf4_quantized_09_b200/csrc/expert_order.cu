// Row order of a batch by expert id: a stable counting sort in one launch.
//
//   order[j]   = the row at place j when the rows stand by id, rows of one id
//                in their own order, ids outside [0, E) behind all others
//   offsets[e] = rows with an id below e; expert e owns places
//                [offsets[e], offsets[e + 1])
//
// One CTA, or a cluster of eight for long batches; each warp takes a contiguous
// piece of the rows, pieces in warp order. Pass 1 counts each warp's ids in
// shared memory: lanes with equal ids find each other by one vote per bit of
// the id, and the lowest of them adds their number (no atomics: a fixed
// result). A scan over the warps, the CTAs of the cluster (through distributed
// shared memory) and the ids turns the counts into first places. Pass 2 writes
// each row to its place: what it needs is in registers for pieces of up to 256
// rows; the ids of longer ones are read again (L2).
//
// Bound by latency: 8 bytes per row move, and two passes, a cluster barrier and a
// scan stand one behind the other; of the issue slots of its eight SMs 40 % are
// used. 32768 ids over 64 experts: 53 us with one CTA and match instructions, 12 us
// with the cluster and votes, 8 us with the keys and places kept; 16 ids over 8
// experts 2.7 us, about what a launch takes. Longer batches stay on eight SMs, and
// from 65536 ids on each id is read twice.
#include <algorithm>

#include "kernels.h"
#include "tiles.cuh"

namespace qlora {

namespace {

constexpr int kMaxWarps = 32;
constexpr int kAhead = 8;  // ids of a lane in flight together
constexpr int kClusterCtas = 8;

// Lanes of the warp whose key equals this one's (whole warp).
__device__ __forceinline__ unsigned same_key(int key, int bits) {
    unsigned same = 0xFFFFFFFFu;
    for (int b = 0; b < bits; ++b) {
        const unsigned v = __ballot_sync(0xFFFFFFFFu, (key >> b) & 1);
        same &= ((key >> b) & 1) ? v : ~v;
    }
    return same;
}

__global__ void __launch_bounds__(kMaxWarps * 32)
    expert_order_kernel(const int* __restrict__ ids, int M, int E, int bits, int* __restrict__ order,
                        int* __restrict__ offsets) {
    extern __shared__ int hist[];  // [warps][E + 1], then the CTA's totals [E + 1]
    __shared__ int warp_sum[kMaxWarps];
    const int kWarps = static_cast<int>(blockDim.x) >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, H = E + 1, tid = static_cast<int>(threadIdx.x);
    const int ctas = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
    int* totals = hist + kWarps * H;
    for (int i = tid; i < kWarps * H; i += kWarps * 32) hist[i] = 0;
    __syncthreads();
    const int pieces = kWarps * ctas;
    const int per = ((M + pieces - 1) / pieces + 31) & ~31;
    const int lo = min((cta * kWarps + warp) * per, M), hi = min(lo + per, M);
    int* mine = hist + warp * H;
    // rows past the piece's end get a key of their own, which counts nothing
    auto key_of = [&](int row) {
        if (row >= hi) return (1 << bits) - 1;
        const int id = __ldg(ids + row);
        return id >= 0 && id < E ? id : E;
    };
    // Pass 1. The keys of a piece of up to 32 kAhead rows, and each row's place
    // among the piece's rows of its id, stay in registers for pass 2.
    int key[kAhead], place[kAhead];
    for (int b = lo; b < hi; b += 32 * kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) key[j] = key_of(b + 32 * j + lane);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int row = b + 32 * j + lane;
            if (row - lane >= hi) break;  // the same for the whole warp
            const unsigned same = same_key(key[j], bits);
            const int first = row < hi ? mine[key[j]] : 0;
            place[j] = first + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (row < hi && lane == __ffs(same) - 1) mine[key[j]] = first + __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    // an id's places by warp, and its total in this CTA
    int total = 0, by_warp[kMaxWarps];
    if (tid < H) {
#pragma unroll
        for (int w = 0; w < kMaxWarps; ++w) by_warp[w] = w < kWarps ? hist[w * H + tid] : 0;
#pragma unroll
        for (int w = 0; w < kMaxWarps; ++w) {
            const int n = by_warp[w];
            by_warp[w] = total;
            total += n;
        }
        totals[tid] = total;
    }
    int before = 0;  // in the CTAs before this one
    if (ctas > 1) {
        cluster_sync();
        if (tid < H) {
            int all = 0;
            for (int c = 0; c < ctas; ++c) {
                int n;
                asm volatile("ld.shared::cluster.s32 %0, [%1];"
                             : "=r"(n)
                             : "r"(mapa_shared(smem_u32(totals + tid), static_cast<uint32_t>(c)))
                             : "memory");
                if (c < cta) before += n;
                all += n;
            }
            total = all;
        }
        cluster_sync();  // no CTA's shared memory is read after this
    }
    const int incl = warp_scan_add(total);
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int s = lane < kWarps ? warp_sum[lane] : 0;
        warp_sum[lane] = warp_scan_add(s) - s;
    }
    __syncthreads();
    if (tid < H) {
        const int start = warp_sum[warp] + incl - total;
        if (cta == 0) offsets[tid] = start;
#pragma unroll
        for (int w = 0; w < kMaxWarps; ++w)
            if (w < kWarps) hist[w * H + tid] = start + before + by_warp[w];
    }
    __syncthreads();
    // Pass 2
    if (per <= 32 * kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int row = lo + 32 * j + lane;
            if (row < hi) order[mine[key[j]] + place[j]] = row;
        }
        return;
    }
    for (int b = lo; b < hi; b += 32 * kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) key[j] = key_of(b + 32 * j + lane);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int row = b + 32 * j + lane;
            const unsigned same = same_key(key[j], bits);
            const int first = row < hi ? mine[key[j]] : 0;
            if (row < hi) order[first + __popc(same & ((1u << lane) - 1u))] = row;
            __syncwarp();
            if (row < hi && lane == __ffs(same) - 1) mine[key[j]] = first + __popc(same);
            __syncwarp();
        }
    }
}

constexpr size_t smem_for(int E, int warps) { return static_cast<size_t>(warps + 1) * (E + 1) * 4; }

}  // namespace

cudaError_t expert_order_init_device() {
    return cudaFuncSetAttribute(expert_order_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem_for(kMaxExperts, kMaxWarps)));
}

cudaError_t launch_expert_order(const int* ids, int M, int E, int* order, int* offsets, cudaStream_t st) {
    static_assert(kMaxExperts + 1 <= kMaxWarps * 32, "one thread per id in the scan");
    if (E < 1 || E > kMaxExperts || M < 0) return cudaErrorInvalidValue;
    // keys 0 .. E, and one more (all ones) for rows that do not exist
    int bits = 1;
    while ((1 << bits) - 1 <= E) ++bits;
    // a cluster once one CTA's lanes would have more than four ids each (the
    // barriers between CTAs cost about a microsecond)
    const int ctas = M > 4 * kMaxWarps * 32 ? kClusterCtas : 1;
    // no more warps than rows or ids to scan need
    const int warps = ctas > 1 ? kMaxWarps : std::min(kMaxWarps, std::max(1, std::max((M + 31) / 32, (E + 32) / 32)));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(warps) * 32);
    cfg.dynamicSmemBytes = smem_for(E, warps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, expert_order_kernel, ids, M, E, bits, order, offsets);
}

}  // namespace qlora
