// Rank-r matmuls of a layer of experts (tcgen05): every expert's adapter over
// its own rows [o_e, o_{e+1}) of the batch.
//
//   down:   sT = s X A_e^T (forward),  sU = s dY B_e (backward)
//   grads:  dA_e = sU^T X,  dB_e = dY^T sT    (fp32, over the expert's rows)
//
// ("waylandz ch.26" 26.2.4 with the adapter chosen by the row's expert.)
//
// Precision. The tensor core takes bf16 operands, and its fp32 accumulator
// truncates: measured on this hardware a sum over 1024 terms is about 1e-6
// low, and the loss grows with the length (2e-5 at 16384). Two measures keep
// the fp32 gradients at fp32 accuracy:
//   - sT and sU leave as sums of bf16 numbers (two for sT, which is kept
//     between the passes; three for sU), each rounding the rest of the one
//     before: 2^-16 and 2^-24 relative at most instead of bf16's 2^-8; the gradients
//     run one UMMA per term into the same accumulator, which costs little
//     beside reading X and dY once;
//   - every 512 reduction elements (128 for sT and sU: at 512 as many of their
//     first terms round the other way as in a plain fp32 sum, at 128 half of
//     those, in the same time) the accumulator is read out and added to fp32
//     registers (round to nearest), two TMEM buffers in turn, so the tensor core
//     never waits for it.
//
// Both kernels read X and dY once (2 bytes per token and column) and are bound by
// the latency of their loads at the bytes in flight that the stages hold: sT of
// 8192 x 4096 22 us (67 MB, 3.1 TB/s); dA and dB of 8 experts of 4096 x 11008 over
// 8192 rows 75 us alone (274 MB, 3.6 TB/s), most of them beside dX's last tiles.
//   warp 0 TMA producer, warp 1 TMEM owner + UMMA issuer, warps 2-5 epilogue.
#include <algorithm>

#include "kernels.h"
#include "tiles.cuh"

namespace qlora {

namespace {

constexpr int kThreads = 192;
constexpr int kFlush = 8;             // 64-deep steps between read-outs of the gradients
constexpr int kDownFlush = 2;         // and of sT and sU
constexpr uint32_t kABytes = 128 * 64 * 2;
constexpr uint32_t kTmemCols = 128;   // two accumulators of up to 64 columns
constexpr int kMaxStages = 8;
constexpr uint32_t kRowBytes = 256;   // one fp32 accumulator row in the reduction buffer

__device__ __forceinline__ uint64_t mn_b_desc(uint32_t addr, int NR) {
    // [64 reduction rows, NR columns] with the NR * 2-byte swizzle: rows of
    // NR * 2 bytes, 8-row groups 16 NR bytes apart, one atom spanning all columns
    const uint32_t layout = NR == 16 ? 6u : (NR == 32 ? 4u : 2u);
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(1u) << 16;
    d |= static_cast<uint64_t>((16u * static_cast<uint32_t>(NR) >> 4) & 0x3FFFu) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(layout) << 61;
    return d;
}

struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_free[2], tail_in, masked, drain;
    uint32_t tmem_slot;
    int abort_flag;
    int tile[4];
};

__device__ __forceinline__ void init_bars(Bars* b, int stages) {
    for (int s = 0; s < stages; ++s) {
        mbar_init(b->full + s, 1);
        mbar_init(b->empty + s, 1);
    }
    for (int p = 0; p < 2; ++p) {
        mbar_init(b->acc_full + p, 1);
        mbar_init(b->acc_free + p, 4);
    }
    mbar_init(&b->tail_in, 1);
    mbar_init(&b->masked, 4);
    mbar_init(&b->drain, 1);
    b->abort_flag = 0;
    fence_mbar_init();
}

// Adds accumulator buffer `chunk & 1` (NR columns) to this thread's row.
__device__ __forceinline__ bool flush_acc(Bars* b, uint32_t tmem, int q, int lane, int NR, int chunk, float (&v)[64],
                                          uint64_t tmo, int* status) {
    const int p = chunk & 1;
    const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(b->acc_full + p, static_cast<uint32_t>(chunk >> 1) & 1u, tmo, status));
    if (!ok) return false;
    tc_fence_after();
#pragma unroll
    for (int c0 = 0; c0 < 64; c0 += 16) {
        if (c0 < NR) {
            uint32_t r[16];
            tmem_ld16(tmem + (static_cast<uint32_t>(q * 32) << 16) + p * 64 + c0, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[c0 + i] += __uint_as_float(r[i]);
        }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(b->acc_free + p);
    return true;
}

// ------------------------------------------------------------------- down --
// One cluster of S CTAs per 128-row tile of an expert; split y takes the
// 64-deep steps y, y + S, ...; partial sums are added in rank order through
// distributed shared memory.
template <bool kBMn>
__global__ void __launch_bounds__(kThreads, 2)
    expert_down(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                const ExpertDownArgs a) {
    asm volatile("griddepcontrol.launch_dependents;");
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars bars;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    clear_words(a.clear, a.clear_words, static_cast<int>(blockIdx.x * gridDim.y + blockIdx.y), static_cast<int>(gridDim.x * gridDim.y));
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int NR = a.NR, S = a.splits, y = static_cast<int>(blockIdx.y);
    const uint32_t b_bytes = static_cast<uint32_t>(NR) * 128u, stage = kABytes + b_bytes;
    const int stages = a.stages;
    const uint64_t tmo = a.timeout_ns;
    if (warp == 0) {
        int e = 0, row0 = 0, rows = 0;
        const bool found = find_row_tile(a.offsets, a.E, static_cast<int>(a.M), 128, static_cast<int>(blockIdx.x), &e, &row0,
                                         &rows);
        if (lane == 0) {
            bars.tile[0] = found ? rows : 0;
            bars.tile[1] = e;
            bars.tile[2] = row0;
            init_bars(&bars, stages);
            tma_prefetch_desc(&tm_a);
            tma_prefetch_desc(&tm_b);
        }
    }
    __syncthreads();
    const int rows = bars.tile[0], e = bars.tile[1], row0 = bars.tile[2];
    if (rows == 0) return;  // past the last tile: the whole cluster
    if (warp == 1) {
        tmem_alloc(&bars.tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_slot;
    volatile int* abort_flag = &bars.abort_flag;
    const int KT = static_cast<int>((a.red + 63) / 64);
    const int steps = y < KT ? (KT - y + S - 1) / S : 0;
    const int chunks = (steps + kDownFlush - 1) / kDownFlush;

    if (warp == 0) {
        if (lane == 0) {
            int i = 0;
            for (; i < steps; ++i) {
                const int s = i % stages;
                if (i >= stages && !mbar_wait(bars.empty + s, static_cast<uint32_t>(i / stages - 1) & 1u, tmo, a.status)) {
                    *abort_flag = 1;
                    break;
                }
                if (*abort_flag) break;
                const int k = (i * S + y) * 64;
                uint8_t* st = smem + s * stage;
                mbar_arrive_expect_tx(bars.full + s, stage);
                tma_load_2d(st, &tm_a, bars.full + s, k, row0);
                if (!kBMn)
                    tma_load_3d(st + kABytes, &tm_b, bars.full + s, k, 0, e);
                else
                    tma_load_3d(st + kABytes, &tm_b, bars.full + s, 0, k, e);
            }
            for (int j = max(0, i - stages); j < i; ++j)
                mbar_wait(bars.full + j % stages, static_cast<uint32_t>(j / stages) & 1u, tmo, nullptr);
        }
        __syncwarp();
    } else if (warp == 1) {
        const bool leader = elect_one();
        const uint32_t idesc = idesc_bf16(128, NR, false, kBMn);
        const uint64_t ad0 = sw128_desc(smem_u32(smem), 16, 1024);
        const uint64_t bd0 = kBMn ? mn_b_desc(smem_u32(smem) + kABytes, NR) : sw128_desc(smem_u32(smem) + kABytes, 16, 1024);
        const uint32_t bk = static_cast<uint32_t>(kBMn ? 16 * NR * 2 : 32) / 16;
        bool ok = true;
        for (int i = 0; ok && i < steps; ++i) {
            const int s = i % stages, chunk = i / kDownFlush, p = chunk & 1;
            if (i % kDownFlush == 0 && chunk >= 2)
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(bars.acc_free + p, static_cast<uint32_t>((chunk >> 1) - 1) & 1u, tmo,
                                                       a.status));
            ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(bars.full + s, static_cast<uint32_t>(i / stages) & 1u, tmo, a.status));
            if (!ok) break;
            tc_fence_after();
            if (leader) {
                const uint64_t ad = ad0 + static_cast<uint32_t>(s) * (stage / 16), bd = bd0 + static_cast<uint32_t>(s) * (stage / 16);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_f16(tmem + p * 64, ad + kk * 2, bd + kk * bk, idesc, (i % kDownFlush > 0 || kk > 0) ? 1u : 0u);
                umma_commit(bars.empty + s);
                if (i % kDownFlush == kDownFlush - 1 || i == steps - 1) umma_commit(bars.acc_full + p);
            }
            __syncwarp();
        }
        if (!ok) *abort_flag = 1;
        if (leader) umma_commit(&bars.drain);
        mbar_wait(&bars.drain, 0u, tmo, nullptr);
        __syncwarp();
    } else {
        const int q = warp & 3, t = q * 32 + lane;
        float v[64];
#pragma unroll
        for (int j = 0; j < 64; ++j) v[j] = 0.0f;
        bool ok = true;
        for (int c = 0; ok && c < chunks; ++c) ok = flush_acc(&bars, tmem, q, lane, NR, c, v, tmo, a.status);
        if (!ok) *abort_flag = 1;
        // this row to the reduction buffer in the first stages (idle: every
        // copy has landed and every UMMA has completed), 16-byte chunk c at
        // t * 256 + ((c ^ (t & 7)) << 4)
        const uint32_t buf = smem_u32(smem) + static_cast<uint32_t>(t) * kRowBytes;
        if (ok) {
#pragma unroll
            for (int c = 0; c < 16; ++c)
                if (4 * c < NR) {
                    const uint32_t w4[4] = {__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]),
                                            __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3])};
                    sts128(buf + ((static_cast<uint32_t>(c) ^ static_cast<uint32_t>(t & 7)) << 4), w4);
                }
        }
    }

    tc_fence_before();
    cluster_sync();
    {
        const int rank = static_cast<int>(cluster_ctarank());
        const int rows_per = 128 / S, cols4 = a.r / 4, T = a.terms;
        const uint32_t buf0 = smem_u32(smem);
        for (int itm = threadIdx.x; itm < rows_per * cols4; itm += kThreads) {
            const int t = rank * rows_per + itm / cols4, c = itm % cols4;
            if (t >= rows) continue;
            const uint32_t off = static_cast<uint32_t>(t) * kRowBytes + ((static_cast<uint32_t>(c) ^ (t & 7)) << 4);
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            for (int s = 0; s < S; ++s) {
                const float4 p = ld_cluster_f4(mapa_shared(buf0 + off, static_cast<uint32_t>(s)));
                x[0] += p.x;
                x[1] += p.y;
                x[2] += p.z;
                x[3] += p.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = __fmul_rn(a.scale, x[j]);
            uint16_t* out = a.out + (static_cast<int64_t>(row0 + t) * T) * a.r + 4 * c;
            for (int k = 0; k < T; ++k) {
                const uint2 o = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
                *reinterpret_cast<uint2*>(out + k * a.r) = o;
                // what this term leaves (exact in fp32); an infinity or a NaN
                // is carried by the first term alone
                const float h[4] = {__uint_as_float(o.x << 16), __uint_as_float(o.x & 0xFFFF0000u), __uint_as_float(o.y << 16),
                                    __uint_as_float(o.y & 0xFFFF0000u)};
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = isfinite(h[j]) ? x[j] - h[j] : 0.0f;
            }
        }
    }
    cluster_sync();  // no CTA leaves while another may still read its shared memory
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A few rows: X A_e^T on the CUDA cores, a CTA per row and eight columns, its
// eight warps splitting the reduction. Bound by the latency of one pass over
// 18 K bytes, with every load of a thread in flight at K = 4096. The matmul
// that depends on this launch gets an SM when this one's CTAs leave it: the
// tensor-core kernel above holds its SMs 10 us (K = 4096) to 17 us (11008).
constexpr int kFewThreads = 256;
__global__ void __launch_bounds__(kFewThreads)
    expert_down_few(const uint16_t* __restrict__ X, const uint16_t* __restrict__ A, const ExpertDownArgs a) {
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ float part[kFewThreads / 32][8];
    clear_words(a.clear, a.clear_words, static_cast<int>(blockIdx.x * gridDim.y + blockIdx.y), static_cast<int>(gridDim.x * gridDim.y));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = static_cast<int>(blockIdx.x), j0 = static_cast<int>(blockIdx.y) * 8;
    int e = 0, row0 = 0, rows = 0;
    // the row's expert: tiles of one row, of which the first stands at offset o_0
    const int first = min(max(__ldg(a.offsets), 0), static_cast<int>(a.M));
    if (row < first || !find_row_tile(a.offsets, a.E, static_cast<int>(a.M), 1, row - first, &e, &row0, &rows)) return;
    const int K8 = static_cast<int>(a.red / 8);
    const uint4* x = reinterpret_cast<const uint4*>(X + static_cast<int64_t>(row) * a.red);
    const uint4* w = reinterpret_cast<const uint4*>(A + (static_cast<int64_t>(e) * a.r + j0) * a.red);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int i = static_cast<int>(threadIdx.x); i < K8; i += kFewThreads) {
        const uint4 xv = __ldg(x + i);
        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
        uint4 wv[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) wv[j] = __ldg(w + static_cast<int64_t>(j) * K8 + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t ww[4] = {wv[j].x, wv[j].y, wv[j].z, wv[j].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[j] = __fmaf_rn(__uint_as_float(xw[k] << 16), __uint_as_float(ww[k] << 16), acc[j]);
                acc[j] = __fmaf_rn(__uint_as_float(xw[k] & 0xFFFF0000u), __uint_as_float(ww[k] & 0xFFFF0000u), acc[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], d);
        if (lane == j) part[warp][j] = acc[j];
    }
    __syncthreads();
    if (warp == 0 && lane < 8) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < kFewThreads / 32; ++i) v += part[i][lane];
        v = __fmul_rn(a.scale, v);
        uint16_t* out = a.out + (static_cast<int64_t>(row) * a.terms) * a.r + j0 + lane;
        for (int k = 0; k < a.terms; ++k) {
            const uint32_t h = pack_bf16x2(v, 0.0f) & 0xFFFFu;
            out[k * a.r] = static_cast<uint16_t>(h);
            const float hf = __uint_as_float(h << 16);
            v = isfinite(hf) ? v - hf : 0.0f;
        }
    }
}

// ------------------------------------------------------------------ grads --
// Tiles of 128 columns of X (dA) or dY (dB) for each expert, taken by
// persistent CTAs, one per SM; the reduction runs over the expert's rows, 64 at
// a time. The terms of sU (sT) stand side by side in memory, and side by side
// they are the UMMA's N (3 r or 2 r columns): every X or dY tile is read once
// from shared memory for all of them, and the epilogue adds the terms' columns.
// The copies of the next tile run ahead of this one's epilogue.
//
// The rows past an expert's end in its last step belong to other experts (or to
// nobody): both operands' copies of them are zeroed in shared memory before the
// UMMA, so whatever they hold, NaN included, adds nothing. An expert without
// rows gets zeros.
constexpr uint32_t kBoxBytes = 64 * 64 * 2;  // 64 rows x 64 columns
constexpr uint32_t kGradTmem = 512;          // two accumulators of up to 192 columns, 256 apart
constexpr uint32_t kGradSmem = 208 * 1024;   // all stages

__global__ void __launch_bounds__(kThreads, 1)
    expert_grads(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_dy,
                 const __grid_constant__ CUtensorMap tm_su, const __grid_constant__ CUtensorMap tm_st,
                 const ExpertGradArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars bars;
    __shared__ int off[kMaxExperts + 1];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int tk = static_cast<int>((a.K + 127) / 128), tn = static_cast<int>((a.N + 127) / 128);
    const int tiles = a.E * (tk + tn), r = a.r;
    const int boxes_u = (a.terms_u * r + 63) / 64, boxes_t = (a.terms_t * r + 63) / 64;
    const uint32_t stage = kABytes + static_cast<uint32_t>(max(boxes_u, boxes_t)) * kBoxBytes;
    const int stages = a.stages;
    const uint64_t tmo = a.timeout_ns;
    // the safe offsets: clamped to [0, M] and to their running maximum
    for (int i = threadIdx.x; i <= a.E; i += kThreads)
        off[i] = min(max(__ldg(a.offsets + i), 0), static_cast<int>(a.M));
    __syncthreads();
    if (warp == 0) {
        int top = 0;
        for (int e0 = 0; e0 <= a.E; e0 += 32) {
            const int v = max(warp_scan_max(e0 + lane <= a.E ? off[e0 + lane] : 0), top);
            __syncwarp();
            if (e0 + lane <= a.E) off[e0 + lane] = v;
            top = __shfl_sync(0xFFFFFFFFu, v, 31);
        }
        if (lane == 0) {
            init_bars(&bars, stages);
            tma_prefetch_desc(&tm_x);
            tma_prefetch_desc(&tm_dy);
            tma_prefetch_desc(&tm_su);
            tma_prefetch_desc(&tm_st);
        }
    }
    if (warp == 1) {
        tmem_alloc(&bars.tmem_slot, kGradTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_slot;
    volatile int* abort_flag = &bars.abort_flag;

    struct GTile {
        int e, c0, row0, m, steps, tail;
        bool is_a;
    };
    auto tile_of = [&](int id) {
        GTile g;
        g.e = id / (tk + tn);
        const int local = id - g.e * (tk + tn);
        g.is_a = local < tk;
        g.c0 = (g.is_a ? local : local - tk) * 128;
        g.row0 = off[g.e];
        g.m = off[g.e + 1] - g.row0;
        g.steps = (g.m + 63) / 64;
        g.tail = g.m - (g.steps - 1) * 64;  // rows of the last step
        return g;
    };

    if (warp == 0) {
        if (lane == 0) {
            int g = 0;
            bool ok = true;
            for (int id = static_cast<int>(blockIdx.x); ok && id < tiles; id += static_cast<int>(gridDim.x)) {
                const GTile t = tile_of(id);
                const int boxes = t.is_a ? boxes_u : boxes_t;
                const CUtensorMap* ta = t.is_a ? &tm_x : &tm_dy;
                const CUtensorMap* tb = t.is_a ? &tm_su : &tm_st;
                for (int i = 0; i < t.steps; ++i, ++g) {
                    const int s = g % stages;
                    if (g >= stages && !mbar_wait(bars.empty + s, static_cast<uint32_t>(g / stages - 1) & 1u, tmo, a.status)) {
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    if (*abort_flag) {
                        ok = false;
                        break;
                    }
                    const int row = t.row0 + i * 64;
                    uint8_t* st = smem + s * stage;
                    mbar_arrive_expect_tx(bars.full + s, kABytes + static_cast<uint32_t>(boxes) * kBoxBytes);
                    tma_load_2d(st, ta, bars.full + s, t.c0, row);
                    tma_load_2d(st + kBoxBytes, ta, bars.full + s, t.c0 + 64, row);
                    for (int k = 0; k < boxes; ++k)
                        tma_load_2d(st + kABytes + k * kBoxBytes, tb, bars.full + s, 64 * k, row);
                }
            }
            for (int j = max(0, g - stages); j < g; ++j)
                mbar_wait(bars.full + j % stages, static_cast<uint32_t>(j / stages) & 1u, tmo, nullptr);
        }
        __syncwarp();
    } else if (warp == 1) {
        const bool leader = elect_one();
        const uint64_t d0 = sw128_desc(smem_u32(smem), kBoxBytes, 1024);
        int g = 0, chunk = 0, masks = 0;
        bool ok = true;
        for (int id = static_cast<int>(blockIdx.x); ok && id < tiles; id += static_cast<int>(gridDim.x)) {
            const GTile t = tile_of(id);
            const int steps = uniform(t.steps), tail = uniform(t.tail);
            const uint32_t idesc = idesc_bf16(128, uniform(((t.is_a ? a.terms_u : a.terms_t) * r + 15) & ~15), true, true);
            for (int i = 0; ok && i < steps; ++i, ++g) {
                const int s = g % stages, p = chunk & 1;
                if (i % kFlush == 0 && chunk >= 2)
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(bars.acc_free + p, static_cast<uint32_t>((chunk >> 1) - 1) & 1u, tmo,
                                                           a.status));
                ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(bars.full + s, static_cast<uint32_t>(g / stages) & 1u, tmo, a.status));
                if (ok && i == steps - 1 && tail < 64) {
                    if (leader) mbar_arrive(&bars.tail_in);  // the epilogue warps zero the rows past the end
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bars.masked, static_cast<uint32_t>(masks) & 1u, tmo, a.status));
                    ++masks;
                }
                if (!ok) break;
                tc_fence_after();
                const bool ends = i % kFlush == kFlush - 1 || i == steps - 1;
                if (leader) {
                    const uint64_t ad = d0 + static_cast<uint32_t>(s) * (stage / 16), bd = ad + kABytes / 16;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_f16(tmem + p * 256, ad + kk * (2048 / 16), bd + kk * (2048 / 16), idesc,
                                 (i % kFlush > 0 || kk > 0) ? 1u : 0u);
                    umma_commit(bars.empty + s);
                    if (ends) umma_commit(bars.acc_full + p);
                }
                __syncwarp();
                if (ends) ++chunk;
            }
        }
        if (!ok) *abort_flag = 1;
        if (leader) umma_commit(&bars.drain);
        mbar_wait(&bars.drain, 0u, tmo, nullptr);
        __syncwarp();
    } else {
        const int q = warp & 3, t = q * 32 + lane;
        int g = 0, chunk = 0, masks = 0;
        bool ok = true;
        for (int id = static_cast<int>(blockIdx.x); ok && id < tiles; id += static_cast<int>(gridDim.x)) {
            const GTile tl = tile_of(id);
            const int T = tl.is_a ? a.terms_u : a.terms_t, boxes = tl.is_a ? boxes_u : boxes_t;
            const int chunks = (tl.steps + kFlush - 1) / kFlush;
            float v[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) v[j] = 0.0f;
            for (int c = 0; ok && c < chunks; ++c, ++chunk) {
                if (c == chunks - 1 && tl.tail < 64) {
                    // the issuer has seen the last step land; its stage's
                    // barrier stays in that phase, so its parity is safe to
                    // read (these warps did not follow the phases before it)
                    const int gl = g + tl.steps - 1, s = gl % stages;
                    ok = __all_sync(0xFFFFFFFFu,
                                    mbar_wait(&bars.tail_in, static_cast<uint32_t>(masks) & 1u, tmo, a.status) &&
                                        mbar_wait(bars.full + s, static_cast<uint32_t>(gl / stages) & 1u, tmo, a.status));
                    if (!ok) break;
                    ++masks;
                    const uint32_t st = smem_u32(smem + s * stage) + static_cast<uint32_t>(tl.tail) * 128u;
                    const uint32_t zero[4] = {0u, 0u, 0u, 0u};
                    const int n = (64 - tl.tail) * 8;  // 16-byte pieces of a box: rows of 128 bytes
                    for (int b = 0; b < 2 + boxes; ++b)
                        for (int x = t; x < n; x += 128) sts128(st + static_cast<uint32_t>(b) * kBoxBytes + x * 16, zero);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.masked);
                }
                const int p = chunk & 1;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(bars.acc_full + p, static_cast<uint32_t>(chunk >> 1) & 1u, tmo, a.status));
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + p * 256;
                for (int k = 0; k < T; ++k) {
#pragma unroll
                    for (int c0 = 0; c0 < 64; c0 += 16) {
                        if (c0 < r) {
                            uint32_t x[16];
                            tmem_ld16(acc + k * r + c0, x);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[c0 + i] += __uint_as_float(x[i]);  // of r = 8, the first eight are used
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.acc_free + p);
            }
            if (!ok) break;
            g += tl.steps;
            if (tl.is_a) {
                if (tl.c0 + t < a.K) {
                    float* out = a.dA + static_cast<int64_t>(tl.e) * r * a.K + tl.c0 + t;
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (j < r) out[static_cast<int64_t>(j) * a.K] = v[j];
                }
            } else if (tl.c0 + t < a.N) {
                float4* out = reinterpret_cast<float4*>(a.dB + (static_cast<int64_t>(tl.e) * a.N + tl.c0 + t) * r);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (4 * j < r) out[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
        }
        if (!ok) *abort_flag = 1;
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kGradTmem);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

constexpr size_t kDownSmem(int NR, int stages) { return static_cast<size_t>(stages) * (kABytes + NR * 128) + 1024; }
constexpr int kDownStages = 4;                 // 72-96 KB: two CTAs per SM

}  // namespace

cudaError_t expert_rank_init_device() {
    cudaError_t e;
    const int down = static_cast<int>(kDownSmem(64, kDownStages));
    if ((e = cudaFuncSetAttribute(expert_down<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, down)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(expert_down<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, down)) != cudaSuccess)
        return e;
    return cudaFuncSetAttribute(expert_grads, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kGradSmem + 1024));
}

cudaError_t launch_expert_down(bool b_mn, const CUtensorMap& act, const CUtensorMap& b, ExpertDownArgs a, int tiles,
                               cudaStream_t st) {
    const int S = a.splits;
    if ((S != 1 && S != 2 && S != 4 && S != 8) || tiles < 1 || a.NR < a.r || a.terms < 1) return cudaErrorInvalidValue;
    a.stages = kDownStages;
    static_assert(kDownStages * kABytes >= 128 * kRowBytes, "the reduction buffer lies in the stages");
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(S));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kDownSmem(a.NR, a.stages);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = static_cast<unsigned>(S);
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return b_mn ? cudaLaunchKernelEx(&cfg, expert_down<true>, act, b, a)
                : cudaLaunchKernelEx(&cfg, expert_down<false>, act, b, a);
}

cudaError_t launch_expert_down_few(const uint16_t* X, const uint16_t* A, const ExpertDownArgs& a, cudaStream_t st) {
    if (a.M < 1 || a.M > kDownFewRows || a.red % 8 != 0 || a.r % 8 != 0) return cudaErrorInvalidValue;
    expert_down_few<<<dim3(static_cast<unsigned>(a.M), static_cast<unsigned>(a.r / 8)), kFewThreads, 0, st>>>(X, A, a);
    return cudaGetLastError();
}

cudaError_t launch_expert_grads(const CUtensorMap& x, const CUtensorMap& dy, const CUtensorMap& su, const CUtensorMap& st_,
                                ExpertGradArgs a, cudaStream_t st) {
    const int boxes = (std::max(a.terms_u, a.terms_t) * a.r + 63) / 64;
    if (a.r < 8 || boxes < 1 || boxes > 3 || a.E < 1 || a.E > kMaxExperts || a.ctas < 1) return cudaErrorInvalidValue;
    a.stages = static_cast<int>(std::min<size_t>(kMaxStages, kGradSmem / (kABytes + boxes * kBoxBytes)));
    const int64_t tiles = static_cast<int64_t>(a.E) * ((a.K + 127) / 128 + (a.N + 127) / 128);
    if (tiles > 0x3FFFFFFF) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(tiles, a.ctas)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = a.stages * (kABytes + boxes * kBoxBytes) + 1024;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, expert_grads, x, dy, su, st_, a);
}

}  // namespace qlora
