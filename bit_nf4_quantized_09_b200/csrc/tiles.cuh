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
// CTA c takes the whole tiles c, c + P, c + 2 P, ... of the full rounds of P
// tiles (neighbouring tiles run at the same time and share rows and weights
// through L2: dealing each CTA one contiguous range of all tiles instead was
// 1.3 times slower on 8192 rows). The tiles left over, fewer than P, would
// leave SMs idle for a round: where it pays, their reduction steps are dealt
// out in equal contiguous ranges, one per CTA. A CTA that has only part of a
// tile's steps leaves its partial sums in a slot of global memory and takes a
// ticket; the last one to come adds the parts in CTA order (whoever it is, the
// order is the same) and writes the tile. Nobody waits for another CTA. Tiles
// of 256 and 512 tokens are always taken whole: a part of 256 KB costs more to
// write and read than a round left partly idle (on single CTAs 722 us whole, 756
// us shared on 8192 rows). Where tiles run on pairs of CTAs, `CTA` is a pair.
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

// TMA copy of a box of one plane of a 3-D tensor.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// The tcgen05 forms of a CTA pair. The pair's UMMA takes the first 128 rows of
// A and the first half of B's rows from the leader's (even) CTA, the others
// from its partner's, at the same shared-memory addresses; each CTA's TMEM gets
// its own 128 rows of D.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {  // a warp of each CTA
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)), "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Arrives on the barrier at this offset in both CTAs.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(0x3))
        : "memory");
}
template <bool kPair>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if (kPair)
        umma_commit_pair(bar);
    else
        umma_commit(bar);
}

// TMA copies into this CTA's shared memory that complete on a barrier of the
// pair's leader (a mapa address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
        "[%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Arrives on a barrier of the pair's leader. What it releases stays in this
// CTA's shared memory and TMEM, where this SM's tensor core meets it, so CTA
// scope is enough; a release at cluster scope waits for the constants' loads in
// flight as well, 1500 to 1900 cycles a step.
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(smem_u32(bar), 0)) : "memory");
}

// N of UMMA h of a pair's tile: its tokens 256 h on, in multiples of 32.
__device__ __forceinline__ int pair_n(int rows, int h) { return min((max(rows - 256 * h, 0) + 31) & ~31, 256); }

// lut_decode8_sx with every permute as the bare instruction: __byte_perm masks
// its selector to three bits a nibble, which here are known to be clear but not
// to the compiler. Integer instructions bound the decoding (22 per 8 weights).
__device__ __forceinline__ void decode8(const Nf4BlockLut& t, uint32_t packed, uint32_t (&out)[4]) {
    const uint32_t idx = packed & 0x77777777u, p4 = packed << 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t sel = h ? idx >> 16 : idx;
        const uint32_t m = prmt_sx(p4, packed, h ? 0xFBEAu : 0xD9C8u);  // 0xFF where the code's top bit is set
        const uint32_t la = prmt_sx(t.lo[0], t.lo[1], sel), lb = prmt_sx(t.lo[2], t.lo[3], sel);
        const uint32_t ha = prmt_sx(t.hi[0], t.hi[1], sel), hb = prmt_sx(t.hi[2], t.hi[3], sel);
        const uint32_t lo = (la & ~m) | (lb & m), hi = (ha & ~m) | (hb & m);
        out[2 * h + 0] = prmt_sx(lo, hi, 0x4051u);
        out[2 * h + 1] = prmt_sx(lo, hi, 0x6273u);
    }
}

struct TileSched {          // in shared memory, one per CTA
    int off[kMaxExperts + 1];   // safe row offsets
    int base[kMaxExperts + 1];  // token tiles of the experts before e; base[E] = all
};

// The words that a thread of a grid zeroes: first, first + stride, ... In 64
// bits: a grid of a CTA per row has more threads than an int counts from 2^23
// rows on.
struct ClearShare {
    int64_t first, stride;
    __host__ __device__ ClearShare(int cta, int ctas, int thread, int threads)
        : first(static_cast<int64_t>(cta) * threads + thread), stride(static_cast<int64_t>(ctas) * threads) {}
};

// CTA `cta` of `ctas` zeroes its share of `words` words: the first kernel of a
// call clears the status word and the tickets for the kernels behind it.
__device__ __forceinline__ void clear_words(int* p, int words, int cta, int ctas) {
    const ClearShare s(cta, ctas, static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x));
    for (int64_t i = s.first; i < words; i += s.stride) p[i] = 0;
}

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
    int id;          // its place in the list
    int k_lo, k_hi;  // reduction steps of this segment
};

// Meeting in memory costs a CTA about 5 us at the end of its range (the parts
// written and fenced, the ticket, the parts read): eight reduction steps. A
// range of fewer than four steps is not worth a CTA.
constexpr int kFixUp = 8, kMinSteps = 4;

// Of the 8-bit product, whose steps are a third as long and whose parts of up to
// 64 rows take longer to join than a few, in its steps; and a quarter of the
// tile's steps, since a stream of weights that fills the memory's rate gains
// nothing by more CTAs. Whole and shared: 8 x 64 x 4096 12.9 and 10.8 us, 64 x 64
// x 4096 15.8 and 17.0, 1 x 22016 x 8192 37.0 and 39.5, 100 x 11008 x 4096 20.0
// and 29.7.
__host__ __device__ inline int int8_fix_up(int M, int steps) { return 16 + (M < 64 ? M : 64) / 4 + steps / 4; }

// The share-out: `tiles` tiles of `steps` reduction steps over P CTAs. Tiles
// below `whole` are taken whole; the steps of the others (units in all) go in
// ranges to Q CTAs, each with at least one step, so that all of the CTAs
// between the first and the last of a tile hold a part of it.
struct Ranges {
    int tiles, steps, P, whole;
    uint32_t Q, units;  // 32 bits: at most P - 1 tiles, and tiles of 65536 steps or more are taken whole
    // share: whether tiles may be shared at all
    __device__ Ranges(int tiles_, int steps_, int ctas, bool share, int fix_up = kFixUp, int min_steps = kMinSteps)
        : tiles(tiles_), steps(steps_), P(ctas) {
        const int rest = tiles % P;
        whole = tiles;
        units = 0;
        Q = 0;
        if (share && rest > 0 && steps < 65536 && P <= 256) {
            const int u = rest * steps;
            const int q = min(P, max(u / min_steps, rest));
            if ((u + q - 1) / q + fix_up < steps) {
                whole = tiles - rest;
                units = static_cast<uint32_t>(u);
                Q = static_cast<uint32_t>(q);
            }
        }
    }
    __device__ int begin(int c) const { return static_cast<int>(static_cast<uint32_t>(c) * units / Q); }
    __device__ int cta_of(int u) const { return static_cast<int>(((static_cast<uint32_t>(u) + 1u) * Q - 1u) / units); }
    // The CTAs that share tile `id`, and the slot in which one of them leaves
    // its part: each touches at most two tiles in part, the one its range
    // begins in and the one it ends in.
    __device__ int first_cta(int id) const { return cta_of((id - whole) * steps); }
    __device__ int last_cta(int id) const { return cta_of((id - whole) * steps + steps - 1); }
    __device__ int slot(int c, int id) const { return 2 * c + (begin(c) >= (id - whole) * steps ? 0 : 1); }
};
static_assert(256ull * 255 * 65536 < (1ull << 32), "32-bit products");

// Walks the segments of CTA c: its whole tiles, then its range. Token tiles
// are multiples of kRound rows.
template <int kRound = 16>
struct SegIter {
    const TileSched& s;
    const Ranges& r;
    int tile, tiles_w, e, u, u1;
    __device__ SegIter(const TileSched& sched, const Ranges& ranges, int c, int tiles_w_)
        : s(sched), r(ranges), tile(c), tiles_w(tiles_w_), e(0), u(0), u1(0) {
        if (static_cast<uint32_t>(c) < r.Q) {
            u = r.begin(c);
            u1 = r.begin(c + 1);
        }
    }
    __device__ void stop() {
        tile = r.whole;
        u = u1;
    }
    __device__ bool next(Tile& out) {
        if (tile < r.whole) {
            out.id = tile;
            out.k_lo = 0;
            out.k_hi = r.steps;
            tile += r.P;
        } else if (u < u1) {
            const int local = u / r.steps;
            out.id = r.whole + local;
            out.k_lo = u - local * r.steps;
            out.k_hi = min(r.steps, out.k_lo + u1 - u);
            u += out.k_hi - out.k_lo;
        } else {
            return false;
        }
        while (out.id >= s.base[e + 1] * tiles_w) ++e;
        const int n = s.base[e + 1] - s.base[e];  // token tiles of this expert, at least 1
        const int local = out.id - s.base[e] * tiles_w;
        const int m = s.off[e + 1] - s.off[e];
        const int per = ((m + n - 1) / n + kRound - 1) & ~(kRound - 1);
        const int j = local % n;
        out.e = e;
        out.w0 = local / n * 256;
        out.row0 = s.off[e] + j * per;
        out.rows = min(per, s.off[e + 1] - out.row0);
        return true;
    }
};

// The tiles a CTA has left a part of (in shared memory; one thread writes).
struct SharedTiles {
    int n;
    int last[2];   // whether this CTA is the last to come, and finishes the tile
    Tile tile[2];
    __device__ void push(const Tile& t) { tile[n++] = t; }
    __device__ void take_tickets(const Ranges& r, int* tickets, bool ok) {
        for (int k = 0; k < n; ++k)
            last[k] = ok && atomicAdd(tickets + tile[k].id, 1) == r.last_cta(tile[k].id) - r.first_cta(tile[k].id);
    }
};

// Adds the parts of a shared tile (rows x 256 words each) in CTA order and
// hands every four columns to `put(token, column, sums)`; `threads` threads,
// this one `t`. The parts lie in slot `slot0` (CTA c0's) and, for the CTAs
// after it, whose ranges begin inside the tile, in slots 2 c. Eight loads per
// thread are in flight (four tokens, two parts).
template <typename T4, typename Put>
__device__ __forceinline__ void add_parts(const void* part, int slot_words, int slot0, int c0, int c1, int rows, int cols,
                                          int t, int threads, Put put) {
    const int nc = 4 * (t & 63);  // threads is a multiple of 64
    if (nc >= cols) return;
    const int tstep = threads >> 6;
    for (int tok = t >> 6; tok < rows; tok += 4 * tstep) {
        T4 v[4];
        memset(v, 0, sizeof(v));
        for (int c = c0; c <= c1; c += 2) {
            T4 x[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (c + j > c1) break;
                const T4* src = reinterpret_cast<const T4*>(static_cast<const uint32_t*>(part) +
                                                            (c + j == c0 ? slot0 : 2 * (c + j)) * slot_words + nc);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (tok + k * tstep < rows) x[j][k] = __ldcg(src + (tok + k * tstep) * 64);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (c + j <= c1) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        v[k].x += x[j][k].x;
                        v[k].y += x[j][k].y;
                        v[k].z += x[j][k].z;
                        v[k].w += x[j][k].w;
                    }
                }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (tok + k * tstep < rows) put(tok + k * tstep, nc, v[k]);
    }
}

// A barrier of `threads` threads (named barrier 1) that also says whether `ok`
// held for all of them.
__device__ __forceinline__ bool all_ok(bool ok, int threads) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, r;\n\tsetp.ne.s32 p, %1, 0;\n\t"
        "bar.red.and.pred r, 1, %2, p;\n\tselp.s32 %0, 1, 0, r;\n\t}"
        : "=r"(r)
        : "r"(ok ? 1 : 0), "r"(threads)
        : "memory");
    return r != 0;
}

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

}  // namespace qlora
