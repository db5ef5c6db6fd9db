// The tile list of the grouped matmuls: rows grouped by expert, ragged.
//
// Row offsets o_0 <= o_1 <= ... <= o_E (device, int32) give expert e the rows
// [o_e, o_{e+1}). Each expert's rows are cut into ceil(rows / cap) token tiles
// of equal size (rounded up to 16, the granularity of the UMMA's N), so an
// expert of 260 rows takes two tiles of 144 and 116 rather than 256 and 4;
// times the 256-row tiles of its weight. The list runs expert by expert, then
// by weight tile, then by token tile: CTAs that run at the same time share a
// weight tile's bytes and an expert's rows through L2.
//
// Offsets are read on the device only, so they are made safe there: clamped to
// [0, M] and to their running maximum. Rows outside [o_0, o_E) belong to no
// tile and are never written.
#pragma once

#include "common.cuh"

namespace qlora {

constexpr int kMaxExperts = 512;

// The UMMA issuers of the grouped kernels run their loop with the whole warp
// and issue under elect_one(). Warp number, loop conditions and tile sizes are
// broadcast (uniform), so that the compiler keeps counters and descriptors in
// uniform registers: as per-thread values each one is moved there before every
// UMMA, which cost about 1000 cycles per 64-deep step of eight UMMAs.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
__device__ __forceinline__ int warp_index() { return uniform(static_cast<int>(threadIdx.x >> 5)); }

// Both phases complete (whole warp, uniform result): one look at each, then
// the bounded waits.
__device__ __forceinline__ bool wait_both(uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1, uint64_t tmo, int* status) {
    const bool r0 = mbar_try_wait(smem_u32(b0), p0), r1 = mbar_try_wait(smem_u32(b1), p1);
    if (__all_sync(0xFFFFFFFFu, r0 && r1)) return true;
    return __all_sync(0xFFFFFFFFu, mbar_wait(b0, p0, tmo, status) && mbar_wait(b1, p1, tmo, status));
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

struct TileSched {          // in shared memory, one per CTA
    int off[kMaxExperts + 1];   // safe row offsets
    int base[kMaxExperts + 1];  // token tiles of the experts before e; base[E] = all
};

// Inclusive scans over a warp.
__device__ __forceinline__ int warp_scan_max(int v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v = max(v, u);
    }
    return v;
}
__device__ __forceinline__ int warp_scan_add(int v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v += u;
    }
    return v;
}

// Builds the schedule; every thread of the CTA takes part, the caller
// synchronises the CTA afterwards. offsets == nullptr: one expert, all M rows.
__device__ __forceinline__ void build_sched(TileSched& s, const int* offsets, int E, int M, int cap) {
    for (int i = threadIdx.x; i <= E; i += blockDim.x) {
        const int raw = offsets ? __ldg(offsets + i) : (i ? M : 0);
        s.off[i] = min(max(raw, 0), M);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int top = 0, tiles = 0;  // carried over chunks of 32 experts
        for (int e0 = 0; e0 <= E; e0 += 32) {
            const int e = e0 + lane;
            int v = warp_scan_max(e <= E ? s.off[e] : 0);
            v = max(v, top);
            int prev = __shfl_up_sync(0xFFFFFFFFu, v, 1);
            if (lane == 0) prev = e0 ? top : v;  // offset e - 1; expert e - 1 owns [prev, v)
            const int n = e <= E ? (v - prev + cap - 1) / cap : 0;
            const int sum = warp_scan_add(n) + tiles;
            __syncwarp();
            if (e <= E) {
                s.off[e] = v;
                s.base[e] = sum;  // tiles of the experts before e
            }
            top = __shfl_sync(0xFFFFFFFFu, v, 31);
            tiles = __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
    }
}

struct Tile {
    int e;           // expert
    int row0, rows;  // its token rows: 1 <= rows <= cap
    int w0;          // first row of the weight tile
};

// Walks the tiles first, first + stride, ... of a launch.
struct TileIter {
    const TileSched& s;
    int t, stride, tiles_w, E, e;
    __device__ TileIter(const TileSched& sched, int first, int stride_, int tiles_w_, int E_)
        : s(sched), t(first), stride(stride_), tiles_w(tiles_w_), E(E_), e(0) {}
    __device__ bool next(Tile& out) {
        if (t >= s.base[E] * tiles_w) return false;
        while (t >= s.base[e + 1] * tiles_w) ++e;
        const int n = s.base[e + 1] - s.base[e];  // token tiles of this expert, at least 1
        const int local = t - s.base[e] * tiles_w;
        const int m = s.off[e + 1] - s.off[e];
        const int per = ((m + n - 1) / n + 15) & ~15;
        const int j = local % n;
        out.e = e;
        out.w0 = local / n * 256;
        out.row0 = s.off[e] + j * per;
        out.rows = min(per, s.off[e + 1] - out.row0);
        t += stride;
        return true;
    }
};

// Finds tile `x` of the list of `cap`-row token tiles without keeping the list
// (one warp; per-expert tiles of exactly cap rows, the last one shorter).
// Returns false past the end.
__device__ __forceinline__ bool find_row_tile(const int* offsets, int E, int M, int cap, int x, int* e_out, int* row0,
                                              int* rows) {
    const int lane = threadIdx.x & 31;
    int top = 0, tiles = 0;
    for (int e0 = 0; e0 <= E; e0 += 32) {
        const int e = e0 + lane;
        int v = warp_scan_max(e <= E ? min(max(__ldg(offsets + e), 0), M) : 0);
        v = max(v, top);
        int prev = __shfl_up_sync(0xFFFFFFFFu, v, 1);
        if (lane == 0) prev = e0 ? top : v;
        const int n = e <= E ? (v - prev + cap - 1) / cap : 0;
        const int end = warp_scan_add(n) + tiles;
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, x < end && x >= end - n);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int first = __shfl_sync(0xFFFFFFFFu, prev, src), last = __shfl_sync(0xFFFFFFFFu, v, src);
            const int local = x - __shfl_sync(0xFFFFFFFFu, end - n, src);
            *e_out = e0 + src - 1;  // the tiles counted at offset e are those of expert e - 1
            *row0 = first + local * cap;
            *rows = min(cap, last - *row0);
            return true;
        }
        top = __shfl_sync(0xFFFFFFFFu, v, 31);
        tiles = __shfl_sync(0xFFFFFFFFu, end, 31);
    }
    return false;
}

// The safe rows [first, last) of expert e (one warp).
__device__ __forceinline__ void expert_rows(const int* offsets, int e, int M, int* first, int* last) {
    const int lane = threadIdx.x & 31;
    int top = 0;
    for (int i = lane; i <= e; i += 32) top = max(top, min(max(__ldg(offsets + i), 0), M));
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    *first = top;
    *last = max(top, min(max(__ldg(offsets + e + 1), 0), M));
}

}  // namespace qlora
