// The expert forward for few rows: Y[m] = X[m] . deq(W_e)^T + sT[m] . B_e^T in
// tiles of up to 16 rows.
//
// With a handful of rows per expert every weight is decoded for a few tokens
// only, and the decoding (what bounds gemm_experts.cu there: 2.75 integer
// instructions per weight, then a trip through shared memory to the UMMA) is
// the whole cost. Here the weights never leave registers: mma.m16n8k16 takes
// them as its A operand straight from the decoder, tokens are its N side (8 or
// 16).
//
// Decoding, exactly w_hat = bf16(fp32(level[code] c')), in two ways side by
// side, since one is bound by shared memory and the other by the integer pipe:
//   - by a table of level pairs: a code byte holds two consecutive weights (the
//     first in the high nibble), entry e is the fp32 pair (level[e >> 4],
//     level[e & 15]). Two weights take a byte permute (the offset), a 64-bit
//     load, one packed multiplication by the block's constant and one
//     conversion to a bf16 pair, the operand register. The table has 16 copies,
//     copy l of entry e at byte 256 e + 8 l: the 16 lanes of each half of a
//     64-bit load meet 32 different banks, and the permute of the code word and
//     8 l is the whole offset. The other 128 bytes of the 256-byte entries hold
//     the stages' block constants.
//   - by byte permutes of the block's 16 products (decode8), as in
//     gemm_experts.cu.
// All of it by table keeps the shared-memory pipe 85 % busy (64 rows over 8
// experts of 4096 x 11008: 94 us), half and half the integer pipe 85 % (also 94
// us); three quarters by table leaves neither the bound alone (91 us).
//
// A warp owns 32 rows of the 256-row weight tile as two 16-row MMA tiles that
// share the token fragments; the second decodes half of its words by permutes.
// A reduction step is four block columns (the codes of 256 rows: one 128-byte x
// 256-row TMA box), and lane (g, q) of a warp owns block q of its rows: the
// products of a block are made once, by one lane. An MMA takes four weights of
// each lane (A slots 2q, 2q + 1, 2q + 8, 2q + 9) and the same columns of the
// tokens; which columns of the step an MMA covers does not matter to the sum.
//
// Producer warps, one per stage, issue the copies and decode the constants.
// Tiles are dealt out as in tiles.cuh: shared tiles meet in global memory, in
// CTA order.
//
// Measured, with the down-projection: two experts of 11008 x 4096 with a row
// each 33 us (47.5 MB, 1.4 TB/s; 42 us by UMMA), 64 rows over 8 experts of 4096
// x 11008 90 us (191.9 MB, 2.1 TB/s; 121 us by UMMA). By timestamps a step takes
// 1.6 us (1.7 in tiles of 16) for 256 x 256 weights (about 3 cycles of the SM for
// 64 weights). Two rows: a CTA's first stage stands 6 us after the first CTA starts
// (11 us where the down-projection held its SM), nine steps take 14.5 us, the
// meeting of shared tiles 2 us. 64 rows: most CTAs start 12 us after the first,
// behind the down-projection's, the first copies take 4.5 us, 37 steps 62 us, the
// meeting 2.5 to 4 us. 16 decoding warps instead of 8 (two groups, steps in turn)
// have 96 registers each and were slower: 37 and 103 us.
#include "kernels.h"
#include "tiles.cuh"

namespace qlora {

namespace {

constexpr int kTilesW = 2;                 // 16-row MMA tiles per warp
constexpr int kWarps = 8;                  // decoding warps: 256 weight rows
constexpr int kTablePairs = 2;             // of a block's four word pairs in the second MMA tile, by table
constexpr int kStep = 4;                   // block columns per reduction step
constexpr uint32_t kTable = 256 * 256;
constexpr uint32_t kCodes = 256 * 32 * kStep;
constexpr int kFixUpSteps = 3, kMinRange = 1;  // as kFixUp and kMinSteps of tiles.cuh, in steps of 256 columns

template <int MT>
struct Lay {
    static constexpr int kCap = 8 * MT;                  // token rows of a tile
    static constexpr int kStages = MT == 1 ? 4 : 3;
    static constexpr int kThreads = (kWarps + kStages) * 32;
    static constexpr uint32_t kXBox = kCap * 128;        // 64 columns of the tokens
    static constexpr uint32_t kStage = kCodes + kStep * kXBox;
    static constexpr uint32_t kOffStage = kTable;
    static constexpr uint32_t kOffSched = kOffStage + kStages * kStage;
    static constexpr uint32_t kOffBar = (kOffSched + sizeof(TileSched) + 63) / 64 * 64;
    static constexpr uint32_t kBytes = kOffBar + 256 + 1024;
};
static_assert(Lay<1>::kBytes <= 227 * 1024 && Lay<2>::kBytes <= 227 * 1024, "shared memory");
static_assert(2 * 4 * 8 + 4 + 4 + sizeof(SharedTiles) <= 256, "barriers");

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

// The bf16 pair of code byte k of w times the constant (twice in cc). The
// table does not change once it is built, so the load may be scheduled freely.
__device__ __forceinline__ uint32_t decode2(uint32_t table, uint32_t lane8, uint32_t w, uint32_t k, uint64_t cc) {
    const uint32_t off = prmt_sx(w, lane8, 0x7704u + (k << 4));
    uint64_t lv, pr;
    asm("ld.shared.b64 %0, [%1];" : "=l"(lv) : "r"(table + off));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(pr) : "l"(lv), "l"(cc));
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(pr));
    return pack_bf16x2(__uint_as_float(lo), __uint_as_float(hi));
}

__device__ __forceinline__ uint64_t twice(float c) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %1};" : "=l"(v) : "f"(c));
    return v;
}

__device__ __forceinline__ float lds_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

// Where stage s holds the four constants of weight row r: in the free half of
// table entry 32 s + r / 8.
__device__ __forceinline__ uint32_t const_at(uint32_t table, int s, int r) {
    return table + static_cast<uint32_t>(32 * s + (r >> 3)) * 256u + 128u + static_cast<uint32_t>(r & 7) * 16u;
}

// Row of its warp tile that fragment row g stands for (g + 8: this + 8): lanes
// 0-15 read rows 0, 2, 4, 6 and lanes 16-31 rows 1, 3, 5, 7, whose 128-byte
// swizzled chunks are disjoint.
__device__ __forceinline__ int frag_row(int g) { return ((g & 3) << 1) | (g >> 2); }

template <int MT, bool kNoDq>
__global__ void __launch_bounds__(Lay<MT>::kThreads, 1)
    expert_gemv(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_codes,
                const __grid_constant__ ExpertGemmArgs a, const __grid_constant__ Nf4Tables tab) {
    using L = Lay<MT>;
    constexpr int S = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    TileSched& sched = *reinterpret_cast<TileSched*>(smem + L::kOffSched);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
    uint64_t* empty = full + 4;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + 4);
    SharedTiles* pending = reinterpret_cast<SharedTiles*>(const_cast<int*>(abort_flag) + 1);
    const uint32_t table = smem_u32(smem);
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int KB = static_cast<int>(a.K / kBlock), N = static_cast<int>(a.N);
    const int steps = (KB + kStep - 1) / kStep;
    const int tiles_w = static_cast<int>((a.N + 255) / 256);
    const uint64_t tmo = a.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + s, 32);       // the lanes of the stage's producer warp
            mbar_init(empty + s, kWarps);
        }
        *abort_flag = 0;
        pending->n = 0;
        fence_mbar_init();
    }
    build_sched(sched, a.offsets, a.E, static_cast<int>(a.M), L::kCap);
    __syncthreads();
    const Ranges ranges(sched.base[a.E] * tiles_w, steps, static_cast<int>(gridDim.x), true, kFixUpSteps, kMinRange);
    SegIter<8> it(sched, ranges, static_cast<int>(blockIdx.x), tiles_w);
    Tile tl;

    if (warp >= kWarps) {
        // ------------------------------------------------------ producers --
        // (warp kWarps + s fills stage s)
        const int s = warp - kWarps;
        if (s == 0 && lane == 0) {
            tma_prefetch_desc(&tm_codes);
            tma_prefetch_desc(&tm_x);
        }
        const float mean = kNoDq ? 0.0f : __ldg(a.c.mean);
        const bool vec = KB % kStep == 0;  // a row's four constants: one aligned word in one group of 256, or a float4
        int k = 0, fills = 0;
        bool ok = true;
        while (ok && uniform(it.next(tl))) {
            for (int kt = tl.k_lo; kt < tl.k_hi; ++kt, ++k) {
                if (k % S != s) continue;
                if (fills > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait_sleep(empty + s, static_cast<uint32_t>(fills - 1) & 1u, tmo,
                                                                          a.status))) {
                    *abort_flag = 1;
                    ok = false;
                    break;
                }
                if (*abort_flag) {
                    ok = false;
                    break;
                }
                uint8_t* st = smem + L::kOffStage + s * L::kStage;
                const int b0 = kt * kStep;
                if (lane == 0) {
                    mbar_expect_tx(full + s, L::kStage);
                    // columns past K and rows past the expert's N or past M read as zeros
                    tma_load_3d(st, &tm_codes, full + s, b0 * 32, tl.w0, tl.e);
#pragma unroll
                    for (int b = 0; b < kStep; ++b)
                        tma_load_2d(st + kCodes + b * L::kXBox, &tm_x, full + s, (b0 + b) * kBlock, tl.row0);
                }
                ++fills;
                // constants of rows lane, lane + 32, ... (past the edges those of
                // the nearest row and column, which reach no output)
#pragma unroll 1
                for (int j0 = 0; j0 < 8; j0 += 4) {
                    float4 c[4];
                    if (vec) {
                        uint32_t qw[4];
                        float sv[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int n = min(tl.w0 + lane + 32 * (j0 + j), N - 1);
                            const uint32_t ib = (static_cast<uint32_t>(tl.e) * static_cast<uint32_t>(N) + n) * KB + b0;  // < 2^32
                            if (kNoDq) {
                                c[j] = __ldg(reinterpret_cast<const float4*>(a.c.absmax + ib));
                            } else {
                                qw[j] = __ldg(reinterpret_cast<const uint32_t*>(a.c.qabsmax + ib));
                                sv[j] = __ldg(a.c.s2 + (ib >> 8));
                            }
                        }
                        if (!kNoDq)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                c[j] = make_float4(__fmaf_rn(e4m3_to_f32(qw[j]), sv[j], mean),
                                                   __fmaf_rn(e4m3_to_f32(qw[j] >> 8), sv[j], mean),
                                                   __fmaf_rn(e4m3_to_f32(qw[j] >> 16), sv[j], mean),
                                                   __fmaf_rn(e4m3_to_f32(qw[j] >> 24), sv[j], mean));
                    } else {
                        uint32_t qv[4][kStep];
                        float sv[4][kStep];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int n = min(tl.w0 + lane + 32 * (j0 + j), N - 1);
                            const uint32_t row = (static_cast<uint32_t>(tl.e) * static_cast<uint32_t>(N) + n) * KB;
#pragma unroll
                            for (int b = 0; b < kStep; ++b) {
                                const uint32_t ib = row + min(b0 + b, KB - 1);
                                if (kNoDq) {
                                    sv[j][b] = __ldg(a.c.absmax + ib);
                                } else {
                                    qv[j][b] = __ldg(a.c.qabsmax + ib);
                                    sv[j][b] = __ldg(a.c.s2 + (ib >> 8));
                                }
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float v[kStep];
#pragma unroll
                            for (int b = 0; b < kStep; ++b)
                                v[b] = kNoDq ? sv[j][b] : __fmaf_rn(e4m3_to_f32(qv[j][b]), sv[j][b], mean);
                            c[j] = make_float4(v[0], v[1], v[2], v[3]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t v[4] = {__float_as_uint(c[j].x), __float_as_uint(c[j].y), __float_as_uint(c[j].z),
                                               __float_as_uint(c[j].w)};
                        sts128(const_at(table, s, lane + 32 * (j0 + j)), v);
                    }
                }
                mbar_arrive(full + s);  // this lane's constants; the copies complete the phase
            }
        }
        // the stage's last copies have landed (also after an abort)
        if (lane == 0 && fills > 0) mbar_wait(full + s, static_cast<uint32_t>(fills - 1) & 1u, tmo, nullptr);
        __syncwarp();
    } else {
        // ------------------------------------------------ decoding and MMA --
        const int g = lane >> 2, q = lane & 3;
        const uint32_t lane8 = 8u * static_cast<uint32_t>(lane & 15);
        const int fr = frag_row(g);
        const int wrow = warp * 16 * kTilesW + fr;  // tile row of fragment row g of MMA tile 0; tile h adds 16 h
        // The lane's words of a block, two by two: pair u = jj ^ q of the block's
        // four at turn jj, an order in which no two lanes of a load meet a bank.
        uint32_t coff[4], xoff[4];
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            const uint32_t u = static_cast<uint32_t>(jj ^ q);
            coff[jj] = static_cast<uint32_t>(wrow) * 128u + (((2u * q + (u >> 1)) ^ static_cast<uint32_t>(fr)) << 4) + ((u & 1u) << 3);
            xoff[jj] = kCodes + static_cast<uint32_t>(q) * L::kXBox + static_cast<uint32_t>(g) * 128u +
                       (((2u * u) ^ static_cast<uint32_t>(g)) << 4);
        }
        // the table, two copies of an entry at a time (while the first copies travel)
        for (int i = threadIdx.x; i < 256 * 8; i += kWarps * 32) {
            const int e = i >> 3;
            const uint32_t v[4] = {__float_as_uint(tab.level[e >> 4]), __float_as_uint(tab.level[e & 15]),
                                   __float_as_uint(tab.level[e >> 4]), __float_as_uint(tab.level[e & 15])};
            sts128(table + static_cast<uint32_t>(e) * 256u + static_cast<uint32_t>(i & 7) * 16u, v);
        }
        bool ok = all_ok(true, kWarps * 32);
        int k = 0;
        while (ok && uniform(it.next(tl))) {
            float acc[kTilesW][MT][4];
#pragma unroll
            for (int h = 0; h < kTilesW; ++h)
#pragma unroll
                for (int t = 0; t < MT; ++t) acc[h][t][0] = acc[h][t][1] = acc[h][t][2] = acc[h][t][3] = 0.0f;
            for (int kt = tl.k_lo; kt < tl.k_hi; ++kt, ++k) {
                const int s = k % S;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(full + s, static_cast<uint32_t>(k / S) & 1u, tmo, a.status));
                if (!ok) break;
                const uint32_t st = table + L::kOffStage + static_cast<uint32_t>(s) * L::kStage;
                // constants of the lane's block, rows fr and fr + 8 of both MMA
                // tiles; a block past K counts as zeros
                float cA[kTilesW], cB[kTilesW];
#pragma unroll
                for (int h = 0; h < kTilesW; ++h) {
                    const uint32_t at = const_at(table, s, wrow + 16 * h) + 4u * q;
                    const bool in = kt * kStep + q < KB;
                    cA[h] = in ? lds_f32(at) : 0.0f;
                    cB[h] = in ? lds_f32(at + 256u) : 0.0f;
                }
                const uint64_t ka = twice(cA[0]), kb = twice(cB[0]), ka1 = twice(cA[1]), kb1 = twice(cB[1]);
                const Nf4BlockLut la = make_block_lut(tab.level, cA[1]), lb = make_block_lut(tab.level, cB[1]);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    const uint2 wa = lds64(st + coff[jj]), wb = lds64(st + coff[jj] + 1024u);
                    const uint2 va = lds64(st + coff[jj] + 2048u), vb = lds64(st + coff[jj] + 2048u + 1024u);
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        uint4 x[MT];
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            // lanes of tokens the tile does not have load nothing and feed zeros
                            x[t] = make_uint4(0u, 0u, 0u, 0u);
                            if (g + 8 * t < tl.rows) x[t] = lds128(((st + xoff[jj]) ^ (16u * w)) + t * 1024u);
                        }
                        const uint32_t ra = w ? wa.y : wa.x, rb = w ? wb.y : wb.x;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t af[4] = {decode2(table, lane8, ra, 2 * i, ka), decode2(table, lane8, rb, 2 * i, kb),
                                                    decode2(table, lane8, ra, 2 * i + 1, ka),
                                                    decode2(table, lane8, rb, 2 * i + 1, kb)};
#pragma unroll
                            for (int t = 0; t < MT; ++t) mma_bf16(acc[0][t], af, i ? x[t].z : x[t].x, i ? x[t].w : x[t].y);
                        }
                        uint32_t oa[4], ob[4];
                        const uint32_t qa = w ? va.y : va.x, qb = w ? vb.y : vb.x;
                        if (jj < kTablePairs) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                oa[i] = decode2(table, lane8, qa, i, ka1);
                                ob[i] = decode2(table, lane8, qb, i, kb1);
                            }
                        } else {
                            decode8(la, qa, oa);
                            decode8(lb, qb, ob);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t af[4] = {oa[2 * i], ob[2 * i], oa[2 * i + 1], ob[2 * i + 1]};
#pragma unroll
                            for (int t = 0; t < MT; ++t) mma_bf16(acc[1][t], af, i ? x[t].z : x[t].x, i ? x[t].w : x[t].y);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + s);
            }
            if (!ok) break;
            if (tl.k_hi == steps) {
                // the rank-r term, by the CTA that has the tile's last step
                asm volatile("griddepcontrol.wait;" ::: "memory");  // sT of the preceding launch
                // (both terms of sT with the same rows of B)
                for (int k1 = 0; k1 < 2 * a.rank_cols; k1 += min(16, a.rank_cols)) {
                    const int term = k1 >= a.rank_cols ? a.rank_cols : 0;
                    const int j0 = k1 - term + 2 * q, j1 = j0 + 8;
                    const bool has1 = j1 < a.rank_cols;
                    uint32_t x0[MT], x1[MT];
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const bool tok = g + 8 * t < tl.rows;
                        const uint16_t* x = a.rank_x + static_cast<int64_t>(tl.row0 + (tok ? g + 8 * t : 0)) * a.rank_ld + term;
                        x0[t] = tok ? __ldcg(reinterpret_cast<const uint32_t*>(x + j0)) : 0u;
                        x1[t] = tok && has1 ? __ldcg(reinterpret_cast<const uint32_t*>(x + j1)) : 0u;
                    }
#pragma unroll
                    for (int h = 0; h < kTilesW; ++h) {
                        const int64_t row = static_cast<int64_t>(tl.e) * N;
                        const uint16_t* bA = a.rank_w + (row + min(tl.w0 + wrow + 16 * h, N - 1)) * a.rank_cols;
                        const uint16_t* bB = a.rank_w + (row + min(tl.w0 + wrow + 16 * h + 8, N - 1)) * a.rank_cols;
                        const uint32_t af[4] = {__ldg(reinterpret_cast<const uint32_t*>(bA + j0)),
                                                __ldg(reinterpret_cast<const uint32_t*>(bB + j0)),
                                                has1 ? __ldg(reinterpret_cast<const uint32_t*>(bA + j1)) : 0u,
                                                has1 ? __ldg(reinterpret_cast<const uint32_t*>(bB + j1)) : 0u};
#pragma unroll
                        for (int t = 0; t < MT; ++t) mma_bf16(acc[h][t], af, x0[t], x1[t]);
                    }
                }
            }
            // acc[h][t][0..1]: row wrow + 16 h, tokens 8t + 2q, + 1; [2..3]: that row + 8
            const bool whole = tl.k_hi - tl.k_lo == steps;
            float* part = a.part + (whole ? 0 : ranges.slot(static_cast<int>(blockIdx.x), tl.id) * a.part_rows * 256);
#pragma unroll
            for (int h = 0; h < kTilesW; ++h)
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = 8 * t + 2 * q + (i & 1), n = wrow + 16 * h + 8 * (i >> 1);
                        if (tok >= tl.rows) continue;
                        if (!whole)
                            part[tok * 256 + n] = acc[h][t][i];
                        else if (tl.w0 + n < N)
                            a.out[static_cast<int64_t>(tl.row0 + tok) * N + tl.w0 + n] =
                                static_cast<uint16_t>(pack_bf16x2(acc[h][t][i], 0.0f));
                    }
            if (!whole && threadIdx.x == 0) pending->push(tl);
        }
        if (!ok) *abort_flag = 1;
        // The tiles shared with other CTAs: their last CTA to come here
        // finishes them. After a wait that ran out nobody does.
        ok = all_ok(ok, kWarps * 32);
        if (ok && pending->n > 0) {
            asm volatile("griddepcontrol.wait;" ::: "memory");  // the launch before has cleared the tickets
            __threadfence();                                     // the parts are visible before the tickets
            all_ok(true, kWarps * 32);
            if (threadIdx.x == 0) pending->take_tickets(ranges, a.tickets, true);
            all_ok(true, kWarps * 32);
            __threadfence();
            for (int j = 0; j < pending->n; ++j) {
                if (!pending->last[j]) continue;
                const Tile p = pending->tile[j];
                uint16_t* out = a.out + static_cast<int64_t>(p.row0) * N + p.w0;
                const int c0 = ranges.first_cta(p.id);
                add_parts<float4>(a.part, a.part_rows * 256, ranges.slot(c0, p.id), c0, ranges.last_cta(p.id), p.rows,
                                  N - p.w0, static_cast<int>(threadIdx.x), kWarps * 32,
                                  [&](int tok, int nc, const float4& v) {
                                      *reinterpret_cast<uint2*>(out + static_cast<int64_t>(tok) * N + nc) =
                                          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                                  });
            }
        }
        __syncwarp();
    }
    // launched as a programmatic dependent, the grid completes only after its primary
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int MT, bool kNoDq>
cudaError_t launch_one(const CUtensorMap& x, const CUtensorMap& codes, const ExpertGemmArgs& a, const Nf4Tables& tab,
                       cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.ctas));
    cfg.blockDim = dim3(Lay<MT>::kThreads);
    cfg.dynamicSmemBytes = Lay<MT>::kBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, expert_gemv<MT, kNoDq>, x, codes, a, tab);
}

template <int MT>
cudaError_t launch_mt(const CUtensorMap& x, const CUtensorMap& codes, const ExpertGemmArgs& a, const Nf4Tables& tab,
                      cudaStream_t st) {
    return a.c.absmax ? launch_one<MT, true>(x, codes, a, tab, st) : launch_one<MT, false>(x, codes, a, tab, st);
}

template <int MT>
cudaError_t opt_in() {
    const cudaError_t e = cudaFuncSetAttribute(expert_gemv<MT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(Lay<MT>::kBytes));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(expert_gemv<MT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(Lay<MT>::kBytes));
}

}  // namespace

cudaError_t expert_gemv_init_device() {
    const cudaError_t e = opt_in<1>();
    if (e != cudaSuccess) return e;
    return opt_in<2>();
}

cudaError_t launch_expert_gemv(const CUtensorMap& x, const CUtensorMap& codes, const ExpertGemmArgs& a, const Nf4Tables& tab,
                               cudaStream_t st) {
    if (a.E < 1 || a.E > kMaxExperts || a.ctas < 1 || a.rank_cols < 8 || a.rank_cols > 64 || a.out_cols != a.N)
        return cudaErrorInvalidValue;
    if (a.cap == 8) return launch_mt<1>(x, codes, a, tab, st);
    if (a.cap == 16) return launch_mt<2>(x, codes, a, tab, st);
    return cudaErrorInvalidValue;
}

}  // namespace qlora
