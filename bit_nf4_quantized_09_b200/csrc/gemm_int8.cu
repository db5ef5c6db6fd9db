// Matrix product in 8-bit integers on tcgen05 (kind::i8), dense or grouped by
// expert:
//
//   Y[m, n] = bf16( xs[m] ws[n] sum_k qx[m, k] qw[n, k] )
//
// qx, xs: the token's row quantised by quantize_rows (one scale per token);
// qw, ws: the weight's (one scale per output channel). This is how the 16-bit
// weight an adapter was merged into is served in fewer bits ("ta-paperlens
// QLoRA explainer", 落とし穴: merging into the 4-bit weight loses the update).
// The int32 sums are exact (K <= 131072 keeps |sum| < 2^31); the roundings are
// the sum's to fp32 (none below 2^24), the scales' product, its product with the
// sum and the bf16 result. Where the scales' product is no normal fp32 number the
// sum is multiplied by one scale after the other (`scaled`).
//
// The weight is the UMMA's M side (256 channels a tile), the tokens its N side,
// as in the NF4 expert matmul, so ragged experts and single tokens pay for the
// tokens they have. Tiles of up to 64 and 256 tokens run on single CTAs, of up
// to 512 on pairs (cta_group::2: 128 channels and half of the tokens each, a
// quarter less to copy for the same work). Persistent CTAs, one per SM:
//   warps 0-15 epilogue (lane = output channel, register = token): a warp reads
//              its 128 tokens' sums, scales and packs them to bf16 in registers
//              and gives the accumulator back before it stores them, so the
//              stores run beside the next tile's UMMAs (a tile's accumulators
//              fill TMEM; 153 us -> 140 us on 4096 x 11008 x 4096)
//   warp 16    TMA producer of token codes (waits for the quantiser's launch,
//              of which this one is the programmatic dependent)
//   warp 17    TMA producer of weight codes (starts at once)
//   warp 18    TMEM owner, UMMA issuer
// The work is dealt out in whole tiles and ranges of reduction steps (tiles.cuh);
// the int32 parts of a tile meet in global memory.
//
// Measured, with the quantiser, among calls that go on for seconds, at the 1.58 and
// 1.52 GHz that the power limit leaves: 4096 x 11008 x 4096 156 us (2.37 Pop/s),
// 8192 rows of 16 experts of 4096 x 4096 152 to 155 us (1.76 Pop/s). In bursts of 40
// ms, at 1.8 to 1.9 GHz, 135 and 132 us (141 and 146 us in tiles of 256). The
// product alone, at 1.84 GHz: 120 us, the tensor pipe 76 % busy. Both are bound by
// the tensor pipe, its clock and the rounds of whole tiles. One token, 22016 x 8192:
// 37 us, 4.9 TB/s, bound by the weight's stream and some 8 us of launches and
// quantising.
#include "kernels.h"
#include "tiles.cuh"

namespace qlora {

namespace {

constexpr int kEpiWarps = 16;
constexpr int kWarpX = 16, kWarpW = 17, kWarpMma = 18;
constexpr int kThreads = (kWarpMma + 1) * 32;
constexpr uint32_t kTmemCols = 512;

template <int CAP>
struct Lay {
    static constexpr bool kPair = CAP == 512;
    static constexpr int kStages = CAP == 512 ? 4 : CAP == 256 ? 3 : 5;
    static constexpr int kBoxRows = CAP == 64 ? 16 : 64;
    static constexpr uint32_t kXHalf = 128 * 128;        // a pair's CTA: 128 tokens of each UMMA
    static constexpr uint32_t kXStage = kPair ? 2 * kXHalf : CAP * 128;
    static constexpr int kRows = kPair ? 128 : 256;      // channels of a CTA
    static constexpr uint32_t kWStage = kRows * 128;
    static constexpr uint32_t kOffW = kStages * kXStage;
    static constexpr uint32_t kOffXs = kOffW + kStages * kWStage;
    static constexpr uint32_t kOffSched = kOffXs + 2048;
    static constexpr uint32_t kOffBar = (kOffSched + sizeof(TileSched) + 63) / 64 * 64;
    static constexpr uint32_t kBytes = kOffBar + 256 + 1024;
};
static_assert(Lay<512>::kBytes <= 227 * 1024 && Lay<256>::kBytes <= 227 * 1024 && Lay<64>::kBytes <= 227 * 1024, "shared memory of one CTA");

__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void umma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor, kind::i8: signed 8-bit A and B (format 1), int32
// accumulator (format 2), both K-major, dense, wrapping.
__device__ __forceinline__ uint32_t idesc_i8(int M, int N) {
    return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// s xs ws, by the scales' product. Where that underflows or overflows, by one
// scale after the other: s xs loses nothing in fp32's subnormals (s is an integer),
// and cannot overflow where xs ws underflows (|s| < 2^31, ws >= 2^-149), so only
// results that leave fp32's range themselves do so, and a sum of zero stays zero.
__device__ __forceinline__ float scaled(float s, float xs, float ws) {
    const float p = xs * ws;
    const bool one = (fabsf(p) < 1.17549435e-38f && xs != 0.0f && ws != 0.0f) || fabsf(p) > 3.40282347e+38f;
    return s * (one ? xs : p) * (one ? ws : 1.0f);
}
// A scale whose product with another such one is normal or zero (or NaN, which stays so).
__device__ __forceinline__ bool middling(float v) {
    return v == 0.0f || !(fabsf(v) < 1.08420217e-19f || fabsf(v) > 9.22337204e+18f);  // 2^-63, 2^63
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 1)
    int8_gemm(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, const Int8GemmArgs a) {
    using L = Lay<CAP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    TileSched& sched = *reinterpret_cast<TileSched*>(smem + L::kOffSched);
    float* xs_s = reinterpret_cast<float*>(smem + L::kOffXs);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
    uint64_t* empty = full + L::kStages;
    uint64_t* acc = empty + L::kStages;
    uint64_t* tmem_free = acc + 1;
    uint64_t* drain = tmem_free + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    SharedTiles* pending = reinterpret_cast<SharedTiles*>(const_cast<int*>(abort_flag) + 1);
    static_assert((2 * L::kStages + 3) * 8 + 8 + sizeof(SharedTiles) <= 256, "barriers");

    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int KT = static_cast<int>((a.K + 127) / 128);
    const int tiles_w = static_cast<int>((a.N + 255) / 256);
    const int crank = L::kPair ? static_cast<int>(cluster_ctarank()) : 0, w_off = crank * L::kRows;
    const int unit = static_cast<int>(blockIdx.x) / (L::kPair ? 2 : 1), units = static_cast<int>(gridDim.x) / (L::kPair ? 2 : 1);
    const uint64_t tmo = a.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(full + s, 2);  // the two producers (+ their bytes)
            mbar_init(empty + s, 1);
        }
        mbar_init(acc, 1);
        mbar_init(tmem_free, kEpiWarps * (L::kPair ? 2 : 1));
        mbar_init(drain, 1);
        *abort_flag = 0;
        pending->n = 0;
        fence_mbar_init();
    }
    if (warp == kWarpMma) {
        if (L::kPair) {
            tmem_alloc_pair(tmem_slot, kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, kTmemCols);
            tmem_relinquish();
        }
    }
    if (warp == kWarpX && lane == 0) {
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_w);
    }
    build_sched(sched, a.offsets, a.E, static_cast<int>(a.M), CAP);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (L::kPair) cluster_sync();  // the partner's barriers are initialised before any remote arrival
    const uint32_t tmem = *tmem_slot;
    const Ranges ranges(sched.base[a.E] * tiles_w, KT, units, CAP == 64, int8_fix_up(static_cast<int>(a.M), KT));
    SegIter<> it(sched, ranges, unit, tiles_w);
    Tile tl;

    if (warp == kWarpX || warp == kWarpW) {
        const bool is_x = warp == kWarpX, leader = elect_one();
        const int cr = uniform(crank);
        if (is_x) asm volatile("griddepcontrol.wait;" ::: "memory");  // the quantised tokens
        int g = 0;
        bool ok = true;
        while (ok && uniform(it.next(tl))) {
            const int rows = uniform(tl.rows), row0 = uniform(tl.row0), w0 = uniform(tl.w0 + w_off), e = uniform(tl.e);
            const int k_lo = uniform(tl.k_lo), k_hi = uniform(tl.k_hi);
            // tokens of each UMMA; of a pair: this CTA's half of them
            const int mine[2] = {L::kPair ? pair_n(rows, 0) / 2 : rows, L::kPair ? pair_n(rows, 1) / 2 : 0};
            const int boxes[2] = {(mine[0] + L::kBoxRows - 1) / L::kBoxRows, (mine[1] + L::kBoxRows - 1) / L::kBoxRows};
            // a pair's leader expects the bytes of both CTAs
            const uint32_t bytes = (is_x ? static_cast<uint32_t>(boxes[0] + boxes[1]) * L::kBoxRows * 128u : L::kWStage) *
                                   (L::kPair ? 2u : 1u);
            for (int k = k_lo; k < k_hi; ++k, ++g) {
                const int s = g % L::kStages;
                if (g >= L::kStages)
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(empty + s, static_cast<uint32_t>(g / L::kStages - 1) & 1u, tmo, a.status));
                if (!ok) *abort_flag = 1;
                if (*abort_flag) ok = false;
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                if (leader) {
                    if (cr == 0) mbar_arrive_expect_tx(full + s, bytes);
                    const uint32_t bar = L::kPair ? mapa_shared(smem_u32(full + s), 0) : 0u;
                    if (is_x) {
#pragma unroll
                        for (int h = 0; h < (L::kPair ? 2 : 1); ++h)
                            for (int b = 0; b < boxes[h]; ++b) {
                                uint8_t* dst = smem + s * L::kXStage + h * L::kXHalf + b * L::kBoxRows * 128;
                                const int row = row0 + 256 * h + cr * mine[h] + b * L::kBoxRows;
                                if (L::kPair)
                                    tma_load_2d_pair(dst, &tm_x, bar, k * 128, row);
                                else
                                    tma_load_2d(dst, &tm_x, full + s, k * 128, row);
                            }
                    } else if (L::kPair) {
                        tma_load_3d_pair(smem + L::kOffW + s * L::kWStage, &tm_w, bar, k * 128, w0, e);
                    } else {
                        tma_load_3d(smem + L::kOffW + s * L::kWStage, &tm_w, full + s, k * 128, w0, e);
                    }
                }
                __syncwarp();
            }
        }
        // no copy still landing when the CTA ends; a partner's complete on the
        // leader's barriers: they have been consumed or, after an abort, land
        // while it waits for what no one signals
        if (cr == 0) {
            for (int j = max(0, g - L::kStages); j < g; ++j)
                mbar_wait(full + j % L::kStages, static_cast<uint32_t>(j / L::kStages) & 1u, tmo, nullptr);
        } else if (!ok) {
            mbar_wait(full, 0u, 1000000u, nullptr);  // 1 ms
        }
        __syncwarp();
    } else if (warp == kWarpMma) {
        const bool leader = elect_one();
        if (L::kPair && crank == 1) it.stop();  // the leader issues for both CTAs
        const uint64_t xd0 = sw128_desc(smem_u32(smem), 16, 1024), wd0 = sw128_desc(smem_u32(smem + L::kOffW), 16, 1024);
        int g = 0, n = 0;
        bool ok = true;
        while (ok && uniform(it.next(tl))) {
            if (n > 0 && !(ok = __all_sync(0xFFFFFFFFu, mbar_wait(tmem_free, static_cast<uint32_t>(n - 1) & 1u, tmo, a.status))))
                break;
            tc_fence_after();
            const int steps = uniform(tl.k_hi - tl.k_lo);
            // two UMMAs at a time: halves of the channels, or of a pair's tokens
            const int rows = uniform(tl.rows);
            const bool two = !L::kPair || rows > 256;
            const uint32_t idesc[2] = {idesc_i8(L::kPair ? 256 : 128, L::kPair ? pair_n(rows, 0) : (rows + 15) & ~15),
                                       idesc_i8(L::kPair ? 256 : 128, L::kPair ? pair_n(rows, 1) : (rows + 15) & ~15)};
            constexpr uint32_t kW2 = L::kPair ? 0 : 16384 / 16, kX2 = L::kPair ? L::kXHalf / 16 : 0;
            for (int i = 0; i < steps; ++i, ++g) {
                const int s = g % L::kStages;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(full + s, static_cast<uint32_t>(g / L::kStages) & 1u, tmo, a.status));
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint64_t xd = xd0 + static_cast<uint32_t>(s) * (L::kXStage / 16);
                    const uint64_t wd = wd0 + static_cast<uint32_t>(s) * (L::kWStage / 16);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (L::kPair) {
                                if (h == 0 || two)
                                    umma_i8_pair(tmem + h * 256, wd + kk * 2, xd + h * kX2 + kk * 2, idesc[h],
                                                 (i > 0 || kk > 0) ? 1u : 0u);
                            } else {
                                umma_i8(tmem + h * 256, wd + h * kW2 + kk * 2, xd + kk * 2, idesc[0],
                                        (i > 0 || kk > 0) ? 1u : 0u);
                            }
                    commit<L::kPair>(empty + s);
                    if (i == steps - 1) commit<L::kPair>(acc);
                }
                __syncwarp();
            }
            ++n;
        }
        if (!ok) *abort_flag = 1;
        if (leader && crank == 0) commit<L::kPair>(drain);
        mbar_wait(drain, 0u, tmo, nullptr);
        __syncwarp();
    } else {
        // ------------------------------------------------------ epilogue --
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the token scales
        const int q = warp & 3, h = (warp >> 2) & 1, part = warp >> 3;
        // channel in the tile; h: a half of a CTA's channels, or of a pair's tokens
        const int nl = L::kPair ? w_off + q * 32 + lane : h * 128 + q * 32 + lane;
        bool ok = true;
        int n = 0;
        while (ok && it.next(tl)) {
            float x = 0.0f;
            if (static_cast<int>(threadIdx.x) < tl.rows) xs_s[threadIdx.x] = x = __ldcg(a.xs + tl.row0 + threadIdx.x);
            const int64_t wrow = static_cast<int64_t>(tl.e) * a.N;
            const float ws = __ldg(a.ws + wrow + min(tl.w0 + nl, static_cast<int>(a.N) - 1));
            // whether every product of two of the tile's scales may be made first
            const bool plain = all_ok(middling(x) && middling(ws), kEpiWarps * 32);
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(acc, static_cast<uint32_t>(n) & 1u, tmo, a.status)) && ok;
            tc_fence_after();
            const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * 256;
            if (CAP != 64 || tl.k_hi - tl.k_lo == KT) {
                // tokens in chunks of 32, every second one this warp's. Two
                // neighbouring lanes swap halves of a token pair: word i of a
                // chunk holds channels nl & ~1, + 1 of token 2 i + (lane & 1).
                constexpr int kChunks = CAP == 64 ? 1 : 4;
                const int tok0 = L::kPair ? 256 * h : 0, toks = min(tl.rows - tok0, 256);
                uint32_t y[kChunks][16];
#pragma unroll
                for (int k = 0; k < kChunks; ++k) {
                    const int c = part * 32 + 64 * k;
                    if (c < toks) {
                        uint32_t r[32];
                        tmem_ld32(trow + c, r);
                        tmem_ld_wait();
                        const float* xs = xs_s + tok0 + c;
                        if (plain) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                r[i] = __float_as_uint(__int2float_rn(static_cast<int>(r[i])) * (xs[i] * ws));
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                r[i] = __float_as_uint(scaled(__int2float_rn(static_cast<int>(r[i])), xs[i], ws));
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float y0 = __uint_as_float(r[i]), y1 = __uint_as_float(r[i + 1]);
                            const float got = __shfl_xor_sync(0xFFFFFFFFu, (lane & 1) ? y0 : y1, 1);
                            y[k][i / 2] = (lane & 1) ? pack_bf16x2(got, y1) : pack_bf16x2(y0, got);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (L::kPair)
                        arrive_leader(tmem_free);
                    else
                        mbar_arrive(tmem_free);
                }
                const int col = tl.w0 + (nl & ~1);
                if (ok && col < a.N) {
                    uint16_t* out = a.Y + static_cast<int64_t>(tl.row0 + tok0) * a.N + col;
#pragma unroll
                    for (int k = 0; k < kChunks; ++k)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int tok = part * 32 + 64 * k + 2 * i + (lane & 1);
                            if (tok < toks) *reinterpret_cast<uint32_t*>(out + tok * a.N) = y[k][i];
                        }
                }
            } else if (CAP == 64) {
                // int32 sums [token][256 channels] to this CTA's slot
                const int slot_ints = a.part_rows * 256;
                int* mine = a.part + ranges.slot(static_cast<int>(blockIdx.x), tl.id) * slot_ints + nl;
                for (int c = part * 32; c < tl.rows; c += 64) {
                    uint32_t r[32];
                    tmem_ld32(trow + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (ok && c + i < tl.rows) mine[(c + i) * 256] = static_cast<int>(r[i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(tmem_free);
                if (threadIdx.x == 0) pending->push(tl);
            }
            ++n;
            // the warps leave together (they meet at barriers), `ok` is the same for
            // all from here to the next wait; this one also ends the reads of this
            // tile's token scales
            ok = all_ok(ok, kEpiWarps * 32);
        }
        // the tiles shared with other CTAs: their last CTA to come here finishes them
        if (CAP == 64 && pending->n > 0) {
            __threadfence();  // the parts are visible before the tickets
            ok = all_ok(ok, kEpiWarps * 32);
            if (threadIdx.x == 0) pending->take_tickets(ranges, a.tickets, ok);
            all_ok(true, kEpiWarps * 32);
            __threadfence();
            for (int k = 0; k < pending->n; ++k) {
                if (!pending->last[k]) continue;
                const Tile p = pending->tile[k];
                uint16_t* out = a.Y + static_cast<int64_t>(p.row0) * a.N + p.w0;
                const float* ws = a.ws + static_cast<int64_t>(p.e) * a.N + p.w0;
                const int c0 = ranges.first_cta(p.id);
                add_parts<int4>(a.part, a.part_rows * 256, ranges.slot(c0, p.id), c0, ranges.last_cta(p.id), p.rows,
                                static_cast<int>(a.N) - p.w0, static_cast<int>(threadIdx.x), kEpiWarps * 32,
                                [&](int tok, int nc, const int4& v) {
                                    const float4 w4 = make_float4(__ldg(ws + nc), __ldg(ws + nc + 1), __ldg(ws + nc + 2),
                                                                  __ldg(ws + nc + 3));
                                    const float x = __ldcg(a.xs + p.row0 + tok);
                                    *reinterpret_cast<uint2*>(out + tok * a.N + nc) =
                                        make_uint2(pack_bf16x2(scaled(__int2float_rn(v.x), x, w4.x), scaled(__int2float_rn(v.y), x, w4.y)),
                                                   pack_bf16x2(scaled(__int2float_rn(v.z), x, w4.z), scaled(__int2float_rn(v.w), x, w4.w)));
                                });
            }
        }
        if (!ok) *abort_flag = 1;
    }

    tc_fence_before();
    __syncthreads();
    if (L::kPair) cluster_sync();  // the leader's UMMAs read and write both CTAs
    if (warp == kWarpMma) {
        tc_fence_after();
        if (L::kPair)
            tmem_dealloc_pair(tmem, kTmemCols);
        else
            tmem_dealloc(tmem, kTmemCols);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------- quantise rows --
// Per row: a = max|x|; code = 127 x / a rounded to the nearest integer, halves
// to even; scale = a / 127. A row of zeros gets codes 0 and scale 0; a row
// that holds a NaN or an infinity gets codes 0 and scale NaN (its products are
// NaN, no other row is touched).
//
// The code is that of the exact quotient: the fp32 product p = x (127 / a) is
// at most 1.6e-5 off, so only a value within 2e-5 of a half j + 1/2 can round
// the wrong way, and there the sign of 127 |x| - (j + 1/2) a decides: both
// products as a rounded number and its remainder (fma), whose differences are
// exact (one look per eight values). Rounding adds and subtracts 1.5 * 2^23
// (its low byte is the code): the conversion instructions run at a quarter of
// the rate.
//
// Bound by reading the row once and writing a byte per element. One CTA per
// row, whose values stay in registers between the two passes over them (4
// vectors of 8 per thread; the rest of a longer row is read again from L2):
// 128 threads up to 4096 columns, 256 above. A warp per row, with no barrier,
// was 1.6 times slower on 8192 x 4096 (too few rows in flight), a CTA loading
// its next row while it works on one 1.3 times (registers).
// 8192 x 4096 from bf16: 17 us alone, 5.9 TB/s.

// Codes of eight values, four to a word.
__device__ __forceinline__ void codes_of(const float (&x)[8], float a, float inv, uint32_t (&w)[2]) {
    uint32_t q[8];
    float off = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float p = x[k] * inv, r = p + 12582912.0f;
        q[k] = __float_as_uint(r);
        off = fmaxf(off, fabsf(p - (r - 12582912.0f)));
    }
    if (off > 0.49998f) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float p = x[k] * inv, ax = fabsf(x[k]);
            if (fabsf(p - ((p + 12582912.0f) - 12582912.0f)) > 0.49998f) {
                const float j = truncf(fabsf(p)), h = j + 0.5f;  // |p| is next to h, on either side
                const float p1 = __fmul_rn(127.0f, ax), h1 = __fmul_rn(h, a);
                const float d = (p1 - h1) + (__fmaf_rn(127.0f, ax, -p1) - __fmaf_rn(h, a, -h1));
                const int ji = static_cast<int>(j);
                const int m = ji + (d > 0.0f || (d == 0.0f && (ji & 1)) ? 1 : 0);
                q[k] = static_cast<uint32_t>(x[k] < 0.0f ? -m : m);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        w[h] = __byte_perm(__byte_perm(q[4 * h], q[4 * h + 1], 0x0040), __byte_perm(q[4 * h + 2], q[4 * h + 3], 0x0040), 0x5410);
}

// Eight consecutive values as they are stored.
template <bool kBf16>
struct Vec8 {
    uint4 w[kBf16 ? 1 : 2];
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        if (kBf16) {
            w[0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at));
        } else {
            const uint4* f = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
            w[0] = __ldg(f);
            w[kBf16 ? 0 : 1] = __ldg(f + 1);
        }
    }
    __device__ __forceinline__ void zero() {
        w[0] = w[kBf16 ? 0 : 1] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t a[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
        if (kBf16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(a[i] << 16);
                v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
            }
        } else {
            const uint4 q = w[kBf16 ? 0 : 1];
            const uint32_t b[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __uint_as_float(a[i]);
                v[4 + i] = __uint_as_float(b[i]);
            }
        }
    }
    // Largest |x| so far as bits of the stored type (bf16 pairwise): a NaN is
    // above an infinity, both above every number.
    __device__ __forceinline__ uint32_t top(uint32_t m) const {
        const uint32_t a[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
        const uint4 q = w[kBf16 ? 0 : 1];
        const uint32_t b[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (kBf16) {
                m = __vmaxu2(m, a[i] & 0x7FFF7FFFu);
            } else {
                m = max(m, a[i] & 0x7FFFFFFFu);
                m = max(m, b[i] & 0x7FFFFFFFu);
            }
        }
        return m;
    }
};

constexpr int kCache = 4;

template <bool kBf16, int TPR>
__global__ void __launch_bounds__(TPR, kBf16 ? 1280 / TPR : 1024 / TPR)
    quantize_rows(const void* X, int64_t K, int8_t* codes, float* scale, int* clear, int clear_n) {
    asm volatile("griddepcontrol.launch_dependents;");
    clear_words(clear, clear_n, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
    const int64_t row = blockIdx.x;
    const int t = threadIdx.x, nv = static_cast<int>(K / 8);
    __shared__ uint32_t part[TPR / 32];
    Vec8<kBf16> c[kCache];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kCache; ++j) {
        const int i = t + j * TPR;
        if (i < nv)
            c[j].load(X, row * K + 8ll * i);
        else
            c[j].zero();
    }
#pragma unroll
    for (int j = 0; j < kCache; ++j) top = c[j].top(top);
    for (int i = t + kCache * TPR; i < nv; i += TPR) {
        Vec8<kBf16> v;
        v.load(X, row * K + 8ll * i);
        top = v.top(top);
    }
    if (kBf16) top = max(top << 16, top & 0x7FFF0000u);  // the larger half, as fp32 bits
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((t & 31) == 0) part[t >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) top = max(top, part[i]);
    const bool bad = top >= 0x7F800000u;
    const float amax = __uint_as_float(top);
    if (t == 0) scale[row] = bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(amax, 127.0f);
    // tiny rows are lifted by 2^64 and huge ones lowered, so that 127 / a, its
    // products and their remainders are normal numbers (what a lowered element
    // loses is far below half a code)
    const float lift = top < 0x2F800000u ? 18446744073709551616.0f
                                         : (top >= 0x6F800000u ? 5.42101086242752217e-20f : 1.0f);
    const float a = amax * lift;
    const bool none = bad || top == 0u;
    const float inv = none ? 0.0f : __fdiv_rn(127.0f, a);
    auto store = [&](int i, const Vec8<kBf16>& vec) {
        uint32_t w[2] = {0u, 0u};
        if (!none) {
            float x[8];
            vec.get(x);
            if (lift != 1.0f) {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] *= lift;
            }
            codes_of(x, a, inv, w);
        }
        *reinterpret_cast<uint2*>(codes + row * K + 8ll * i) = make_uint2(w[0], w[1]);
    };
#pragma unroll
    for (int j = 0; j < kCache; ++j) {
        const int i = t + j * TPR;
        if (i < nv) store(i, c[j]);
    }
    for (int i = t + kCache * TPR; i < nv; i += TPR) {
        Vec8<kBf16> v;
        v.load(X, row * K + 8ll * i);
        store(i, v);
    }
}

template <bool kBf16, int TPR>
cudaError_t launch_quantize(const void* X, int64_t rows, int64_t K, int8_t* codes, float* scale, int* clear, int clear_n,
                            cudaStream_t st) {
    quantize_rows<kBf16, TPR><<<static_cast<unsigned>(rows), TPR, 0, st>>>(X, K, codes, scale, clear, clear_n);
    return cudaGetLastError();
}

template <int CAP>
cudaError_t launch_one(const CUtensorMap& x, const CUtensorMap& w, const Int8GemmArgs& a, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Lay<CAP>::kBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = Lay<CAP>::kPair ? 2 : 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (Lay<CAP>::kPair) cfg.gridDim.x &= ~1u;
    return cudaLaunchKernelEx(&cfg, int8_gemm<CAP>, x, w, a);
}

}  // namespace

cudaError_t int8_init_device() {
    cudaError_t e = cudaFuncSetAttribute(int8_gemm<256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(Lay<256>::kBytes));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(int8_gemm<512>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(Lay<512>::kBytes));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(int8_gemm<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(Lay<64>::kBytes));
}

cudaError_t launch_int8_gemm(const CUtensorMap& x, const CUtensorMap& w, const Int8GemmArgs& a, cudaStream_t st) {
    if (a.E < 1 || a.E > kMaxExperts || a.ctas < 2 || (a.cap != 64 && a.cap != 256 && a.cap != 512))
        return cudaErrorInvalidValue;
    if (a.cap == 512) return launch_one<512>(x, w, a, st);
    return a.cap == 256 ? launch_one<256>(x, w, a, st) : launch_one<64>(x, w, a, st);
}

cudaError_t launch_quantize_rows(const void* X, bool bf16, int64_t rows, int64_t K, int8_t* codes, float* scale,
                                 int* clear, int clear_n, cudaStream_t st) {
    if (rows < 1 || rows > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (K <= 4096)
        return bf16 ? launch_quantize<true, 128>(X, rows, K, codes, scale, clear, clear_n, st)
                    : launch_quantize<false, 128>(X, rows, K, codes, scale, clear, clear_n, st);
    return bf16 ? launch_quantize<true, 256>(X, rows, K, codes, scale, clear, clear_n, st)
                : launch_quantize<false, 256>(X, rows, K, codes, scale, clear, clear_n, st);
}

}  // namespace qlora
