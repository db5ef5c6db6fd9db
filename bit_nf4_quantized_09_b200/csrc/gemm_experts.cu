// Dequant-fused NF4 matmuls over rows grouped by expert (tcgen05 + TMEM + TMA).
//
//   forward:  Y[m]  = X[m] . deq(W_e)^T + sT[m] . B_e^T     W_e: [N, K]
//   dX:       dX[m] = dY[m] . deq(W_e)  + sU[m] . A_e       for the rows m of expert e
//
// The experts' weights are one NF4 weight of E N rows; a stack of frozen 4-bit
// experts, each with an adapter, is QLoRA's layer with the weight chosen per
// token ("ta-paperlens QLoRA explainer", 勾配は実際どこへ行くのか: every matmul
// restores the 4-bit blocks it needs to BF16 on the spot).
//
// Operands. The weight is the UMMA's M side (256 output columns a tile) and the
// tokens its N side (a multiple of 16, of 32 on pairs), so a tile costs what its
// expert's rows cost: an expert with 40 rows runs N = 48. The rank-r term (sT .
// B_e^T, sU . A_e) is two more reduction steps of the same accumulators, their
// operands loaded by TMA: the bf16 rounding of sT or sU, then that of what it
// leaves. How far one rounding shows in the result depends on the adapter's part
// of it and not on the shapes, so both steps always run (2^-16 of |sT| |B|
// at most instead of 2^-8; one step of 66 at K = 4096).
//
// Tiles of up to 64 tokens run on single CTAs, two UMMAs of M = 128 at a time.
// Tiles of up to 256 or 512 tokens run on pairs of CTAs (a cluster of two on
// neighbouring SMs, cta_group::2): each CTA decodes 128 of the 256 weight rows
// and holds half of the tokens, and one UMMA of M = 256 reads both CTAs' shared
// memory, so a weight is decoded once for all tokens of the tile. The leader
// issues for both; copies and decoders of both CTAs arrive on its barriers.
//
// Roles of a persistent CTA (one per SM, 19 warps):
//   warps 0-15  dequantisers in four groups of four that take the reduction
//               steps in turn (64-weight blocks, the exact w_hat =
//               bf16(level c') through the per-block byte tables); then the
//               epilogue
//   warp 16     TMA producer of the token tiles
//   warp 17     TMA producer of the packed codes
//   warp 18     TMEM owner, UMMA issuer
// The producers and the issuer run on warp-uniform values and issue under
// elect_one(): from one lane of a divergent branch a step of copies cost 570
// cycles (8192 rows, with one rank-r step, 663 us, 635 us without).
// Block constants are read from the stored form by the threads that use them;
// no transposed copy of an expert stack's constants is written, most of which
// few tokens would not use.
//
// Bounds, with the down-projection. 8192 rows over 8 experts of 11008 x 4096
// (r = 64): 645 us, 1170 TFLOP/s (613 us in the first calls, before the clock falls
// to the 1.48 GHz that the power limit leaves; 654 us after seconds of them), the
// tensor pipe 81 % busy; on single CTAs, which decode each weight twice as often,
// 715 us (ALU pipe 66 % busy, tensor pipe 68 %). dX of 4096 x 11008: 533 us at 1.59
// GHz, of 720 to 728 for the backward. 1543 rows over 13 experts of 2056 x 4096: 65
// us, bound by decoding (a step of 128 x 64 weights per CTA every 0.35 us, the ALU
// pipe 61 % busy). 160 rows over 8 experts of 4096 x 4096 (tiles of 64): 52 us, a
// step of 256 x 64 weights every 0.67 us.
//
// The work is dealt out in whole tiles and ranges of reduction steps (tiles.cuh);
// parts of a tile meet in global memory, in a fixed order: results are bitwise
// reproducible.
#include "kernels.h"
#include "tiles.cuh"

namespace qlora {

namespace {

constexpr int kDeqWarps = 16;
constexpr int kGroups = 4, kGroupWarps = 4;
constexpr int kWarpX = 16, kWarpC = 17, kWarpMma = 18;
constexpr int kThreads = (kWarpMma + 1) * 32;
constexpr uint32_t kTmemCols = 512;
constexpr int kRankSteps = 2;  // the first two terms of sT or sU

// Shared memory by token capacity.
template <int CAP>
struct Lay {
    static constexpr bool kPair = CAP >= 256;
    static constexpr int kRows = kPair ? 128 : 256;        // weight rows of a CTA
    static constexpr int kP = CAP == 256 ? 6 : 4;          // operand (token and weight) stages
    static constexpr int kPC = 4;                          // code stages
    static constexpr int kBoxRows = kPair ? 64 : 16;       // token rows per TMA box
    static constexpr uint32_t kXHalf = 128 * 128;          // a pair's CTA: 128 tokens of each UMMA
    static constexpr uint32_t kXStage = kPair ? CAP / 256 * kXHalf : CAP * 128;
    static constexpr uint32_t kWStage = kRows * 64 * 2;
    static constexpr uint32_t kCStage = kRows * 64 / 2;    // packed codes
    static constexpr uint32_t kOffW = kP * kXStage;
    static constexpr uint32_t kOffC = kOffW + kP * kWStage;
    static constexpr uint32_t kOffSched = kOffC + kPC * kCStage;
    static constexpr uint32_t kOffBar = (kOffSched + sizeof(TileSched) + 63) / 64 * 64;
    static constexpr uint32_t kBytes = kOffBar + 512 + 1024;
};
static_assert(Lay<512>::kBytes <= 227 * 1024 && Lay<256>::kBytes <= 227 * 1024 && Lay<64>::kBytes <= 227 * 1024, "shared memory of one CTA");
// Code stages are a ring over all reduction steps, but each group waits on
// barriers of its own (two, by the parity of its steps): it has not seen the
// ring's other steps, and a phase parity is only safe to one who has seen the
// phase before. Two steps of one barrier lie at least four reduction steps
// apart (at the least when half of the steps are rank-r steps, two by two), so
// with at most four stages the first has been consumed before the second is
// loaded.
// Operand stages need no such thing: before a group takes stage s for step g it
// has waited for the UMMAs of step g - 4 - kP, so with kP >= 4 the phase before
// is over.
static_assert(Lay<512>::kPC <= 4 && Lay<256>::kPC <= 4 && Lay<64>::kPC <= 4, "code stages");
static_assert(Lay<512>::kP >= kGroups && Lay<256>::kP >= kGroups && Lay<64>::kP >= kGroups, "operand stages");

__device__ __forceinline__ void umma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <bool kTransW, bool kNoDq, int CAP>
__global__ void __launch_bounds__(kThreads, 1)
    expert_gemm(const __grid_constant__ CUtensorMap tm_act, const __grid_constant__ CUtensorMap tm_codes,
                const __grid_constant__ CUtensorMap tm_lact, const __grid_constant__ CUtensorMap tm_lw,
                const ExpertGemmArgs a, const Nf4Tables tab) {
    using L = Lay<CAP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    TileSched& sched = *reinterpret_cast<TileSched*>(smem + L::kOffSched);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);  // tokens and weights of a step
    uint64_t* empty = full + L::kP;
    uint64_t* c_full = empty + L::kP;
    uint64_t* c_empty = c_full + 2 * kGroups;
    uint64_t* acc = c_empty + L::kPC;
    uint64_t* tmem_free = acc + 1;
    uint64_t* drain = tmem_free + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    SharedTiles* pending = reinterpret_cast<SharedTiles*>(const_cast<int*>(abort_flag) + 1);
    static_assert((2 * L::kP + 2 * kGroups + L::kPC + 3) * 8 + 8 + sizeof(SharedTiles) <= 512, "barriers");

    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int KT = static_cast<int>((a.red + 63) / 64);
    const int crank = L::kPair ? static_cast<int>(cluster_ctarank()) : 0;
    const int unit = static_cast<int>(blockIdx.x) / (L::kPair ? 2 : 1), units = static_cast<int>(gridDim.x) / (L::kPair ? 2 : 1);
    const int tiles_w = static_cast<int>((a.out_cols + 255) / 256);
    const uint64_t tmo = a.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kP; ++s) {
            mbar_init(full + s, 1 + kGroupWarps * (L::kPair ? 2 : 1));  // the token producer and the decoders
            mbar_init(empty + s, 1);
        }
        for (int s = 0; s < 2 * kGroups; ++s) mbar_init(c_full + s, 1);
        for (int s = 0; s < L::kPC; ++s) mbar_init(c_empty + s, kGroupWarps);
        mbar_init(acc, 1);
        mbar_init(tmem_free, kDeqWarps * (L::kPair ? 2 : 1));
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
        tma_prefetch_desc(&tm_act);
        tma_prefetch_desc(&tm_lact);
        tma_prefetch_desc(&tm_codes);
        tma_prefetch_desc(&tm_lw);
    }
    build_sched(sched, a.offsets, a.E, static_cast<int>(a.M), CAP);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (L::kPair) cluster_sync();  // the partner's barriers are initialised before any remote arrival
    const uint32_t tmem = *tmem_slot;
    const Ranges ranges(sched.base[a.E] * tiles_w, KT, units, !L::kPair);
    SegIter<> it(sched, ranges, unit, tiles_w);
    Tile tl;
    // steps of a segment: its reduction steps, and the rank-r steps behind a tile's last
    auto steps_of = [&](const Tile& s) { return s.k_hi - s.k_lo + (s.k_hi == KT ? kRankSteps : 0); };

    if (warp == kWarpX) {
        // ------------------------------------------- token-tile producer --
        const bool leader = elect_one();
        const int cr = uniform(crank);
        int g = 0;
        bool waited = false, ok = true;
        while (ok && uniform(it.next(tl))) {
            // of a pair: this CTA's half of each UMMA's tokens
            const int rows = uniform(tl.rows), row0 = uniform(tl.row0), k_lo = uniform(tl.k_lo);
            const int nk = uniform(tl.k_hi) - k_lo, steps = uniform(steps_of(tl));
            const int mine[2] = {L::kPair ? pair_n(rows, 0) / 2 : rows, CAP == 512 ? pair_n(rows, 1) / 2 : 0};
            const int boxes[2] = {(mine[0] + L::kBoxRows - 1) / L::kBoxRows, (mine[1] + L::kBoxRows - 1) / L::kBoxRows};
            // the leader expects the bytes of both CTAs of a pair
            const uint32_t bytes = static_cast<uint32_t>(boxes[0] + boxes[1]) * L::kBoxRows * 128u * (L::kPair ? 2u : 1u);
            auto load = [&](const CUtensorMap* map, int s, int x) {
                if (!leader) return;
                if (cr == 0) mbar_arrive_expect_tx(full + s, bytes);
#pragma unroll
                for (int h = 0; h < (CAP == 512 ? 2 : 1); ++h)
                    for (int b = 0; b < boxes[h]; ++b) {
                        uint8_t* dst = smem + s * L::kXStage + h * L::kXHalf + b * L::kBoxRows * 128;
                        const int row = row0 + 256 * h + cr * mine[h] + b * L::kBoxRows;
                        if (L::kPair)
                            tma_load_2d_pair(dst, map, mapa_shared(smem_u32(full + s), 0), x, row);
                        else
                            tma_load_2d(dst, map, full + s, x, row);
                    }
            };
            for (int i = 0; i < steps; ++i, ++g) {
                const int s = g % L::kP;
                if (g >= L::kP) ok = __all_sync(0xFFFFFFFFu, mbar_wait(empty + s, static_cast<uint32_t>(g / L::kP - 1) & 1u, tmo,
                                                                       a.status));
                if (!ok) *abort_flag = 1;
                if (*abort_flag) ok = false;
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                if (i < nk) {
                    load(&tm_act, s, (k_lo + i) * 64);
                } else {
                    // sT or sU of the preceding launch, of which this one may
                    // be a programmatic dependent
                    if (!waited) {
                        asm volatile("griddepcontrol.wait;" ::: "memory");
                        // behind dX come the gradients, which read sU too
                        asm volatile("griddepcontrol.launch_dependents;");
                    }
                    waited = true;
                    // the columns behind a term's meet zeros of the adapter's tile
                    load(&tm_lact, s, (i - nk) * a.rank_cols);
                }
                __syncwarp();
            }
        }
        // no copy still landing when the CTA ends; a partner's complete on the
        // leader's barriers: they have been consumed or, after an abort, land
        // while it waits for what no one signals
        if (cr == 0) {
            for (int j = max(0, g - L::kP); j < g; ++j)
                mbar_wait(full + j % L::kP, static_cast<uint32_t>(j / L::kP) & 1u, tmo, nullptr);
        } else if (!ok) {
            mbar_wait(full, 0u, 1000000u, nullptr);  // 1 ms
        }
        __syncwarp();
    } else if (warp == kWarpC) {
        // ------------------------------------------------- code producer --
        const bool leader = elect_one();
        int g = 0, g0 = 0;
        uint32_t par = 0;  // per group, parity of its reduction steps so far
        bool ok = true;
        while (ok && uniform(it.next(tl))) {
            const int k_lo = uniform(tl.k_lo), nk = uniform(tl.k_hi) - k_lo, e = uniform(tl.e);
            const int w0 = uniform(tl.w0 + crank * L::kRows);
            for (int i = 0; i < nk; ++i, ++g) {
                const int s = g % L::kPC, G = (g0 + i) & (kGroups - 1);
                uint64_t* bar = c_full + 2 * G + ((par >> G) & 1u);
                if (g >= L::kPC) ok = __all_sync(0xFFFFFFFFu, mbar_wait(c_empty + s, static_cast<uint32_t>(g / L::kPC - 1) & 1u, tmo,
                                                                        a.status));
                if (!ok) *abort_flag = 1;
                if (*abort_flag) ok = false;
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const int kt = k_lo + i;
                par ^= 1u << G;
                if (leader) {
                    mbar_arrive_expect_tx(bar, L::kCStage);
                    // rows past the expert's N and columns past K read as zeros
                    if (!kTransW)
                        tma_load_3d(smem + L::kOffC + s * L::kCStage, &tm_codes, bar, kt * 32, w0, e);
                    else
                        tma_load_3d(smem + L::kOffC + s * L::kCStage, &tm_codes, bar, w0 / 2, kt * 64, e);
                }
                __syncwarp();
            }
            g0 += uniform(steps_of(tl));
        }
        // after an abort copies may still be landing: every stage's last copy is
        // over once its barrier has been consumed, or (bounded) once the time
        // limit has passed
        if (!ok)
            for (int j = max(0, g - L::kPC); j < g; ++j)
                mbar_wait(c_empty + j % L::kPC, static_cast<uint32_t>(j / L::kPC) & 1u, tmo, nullptr);
        __syncwarp();
    } else if (warp == kWarpMma) {
        // ----------------------------------------------------------- MMA --
        const bool leader = elect_one();
        if (L::kPair && crank == 1) {
            it.stop();  // the leader issues for both CTAs
        }
        // descriptors of stage 0; later stages and steps add their byte offset / 16
        const uint64_t xd0 = sw128_desc(smem_u32(smem), 16, 1024);
        const uint64_t wd0 = kTransW ? sw128_desc(smem_u32(smem + L::kOffW), 8192, 1024)
                                     : sw128_desc(smem_u32(smem + L::kOffW), 16, 1024);
        constexpr uint32_t kWk = (kTransW ? 2048 : 32) / 16;
        auto mma = [](uint32_t d, uint64_t wd, uint64_t xd, uint32_t idesc, uint32_t acc_) {
            if (L::kPair)
                umma_f16_pair(d, wd, xd, idesc, acc_);
            else
                umma_f16(d, wd, xd, idesc, acc_);
        };
        int g = 0, n = 0;
        bool ok = true;
        while (ok && uniform(it.next(tl))) {
            if (n > 0 && !(ok = __all_sync(0xFFFFFFFFu, mbar_wait(tmem_free, static_cast<uint32_t>(n - 1) & 1u, tmo, a.status))))
                break;
            tc_fence_after();
            const int nk = uniform(tl.k_hi - tl.k_lo), steps = uniform(steps_of(tl));
            // two UMMAs at a time: halves of the weight rows, or of a pair's tokens
            const int rows = uniform(tl.rows);
            const bool two = CAP == 64 || (CAP == 512 && rows > 256);
            const uint32_t idesc[2] = {idesc_bf16(L::kPair ? 256 : 128, L::kPair ? pair_n(rows, 0) : (rows + 15) & ~15, kTransW, false),
                                       idesc_bf16(L::kPair ? 256 : 128, L::kPair ? pair_n(rows, 1) : (rows + 15) & ~15, kTransW, false)};
            // the second UMMA's operands, behind the first's
            constexpr uint32_t kW2 = L::kPair ? 0 : 16384 / 16, kX2 = L::kPair ? L::kXHalf / 16 : 0;
            for (int i = 0; i < steps; ++i, ++g) {
                const int s = g % L::kP;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(full + s, static_cast<uint32_t>(g / L::kP) & 1u, tmo, a.status));
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint64_t xd = xd0 + static_cast<uint32_t>(s) * (L::kXStage / 16);
                    const uint64_t wd = wd0 + static_cast<uint32_t>(s) * (L::kWStage / 16);
                    if (i < nk) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (h == 0 || two)
                                    mma(tmem + h * 256, wd + h * kW2 + kk * kWk, xd + h * kX2 + kk * 2, idesc[h],
                                        (i > 0 || kk > 0) ? 1u : 0u);
                    } else {
                        for (int kk = 0; kk < (a.rank_cols + 15) / 16; ++kk)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (h == 0 || two) mma(tmem + h * 256, wd + h * kW2 + kk * kWk, xd + h * kX2 + kk * 2, idesc[h], 1u);
                    }
                    commit<L::kPair>(empty + s);
                    if (i == steps - 1) commit<L::kPair>(acc);
                }
                __syncwarp();
            }
            ++n;
        }
        if (!ok) *abort_flag = 1;
        // no UMMA in flight when the TMEM is freed
        if (leader && crank == 0) commit<L::kPair>(drain);
        mbar_wait(drain, 0u, tmo, nullptr);
        __syncwarp();
    } else {
        // ---------------------------------------- dequantise, then epilogue --
        const int G = warp >> 2;            // group, and its weight stage
        const int t = threadIdx.x & 127;    // the thread's two 64-weight blocks of a step: t and t + 128
        const bool leader = t == 0;
        const int q = warp & 3, h = (warp >> 2) & 1, part = warp >> 3;
        // Block constants come from the stored form in global memory, loaded
        // one step of this group (four of the CTA) ahead as they stand: E4M3
        // code and second-level scale, or the fp32 constant. `pit`, `ptl` and
        // `pi` walk that step's position.
        const int KB = static_cast<int>(a.K / kBlock);
        const float mean = kNoDq ? 0.0f : __ldg(a.c.mean);
        SegIter<> pit(sched, ranges, unit, tiles_w);
        constexpr int kU = L::kRows / 128;  // blocks of a thread
        const int w_off = crank * L::kRows;
        Tile ptl;
        int pi = G;
        bool plive = pit.next(ptl);
        uint32_t raw_q[kU] = {};
        float raw_s[kU] = {};
        auto load_constants = [&]() {
            while (plive && pi >= steps_of(ptl)) {
                pi -= steps_of(ptl);
                plive = pit.next(ptl);
            }
            if (!plive || pi >= ptl.k_hi - ptl.k_lo) return;  // nothing left, or the rank-r step
            const int kt = ptl.k_lo + pi;
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                // weight row n and k-block of block u; past the edges of the
                // expert's weight the nearest one inside (not used: codes 0
                // there meet zeros of dY or columns that are not written)
                const int n = min(kTransW ? kt * 64 + (t & 63) : ptl.w0 + w_off + t + 128 * u, static_cast<int>(a.N) - 1);
                const int kb = min(kTransW ? (ptl.w0 + w_off) / kBlock + (t >> 6) + 2 * u : kt, KB - 1);
                const uint32_t ib = (static_cast<uint32_t>(ptl.e) * static_cast<uint32_t>(a.N) + n) * KB + kb;  // < 2^32
                if (kNoDq) {
                    raw_s[u] = __ldg(a.c.absmax + ib);
                } else {
                    raw_q[u] = __ldg(a.c.qabsmax + ib);
                    raw_s[u] = __ldg(a.c.s2 + (ib >> 8));
                }
            }
        };
        load_constants();
        // this warp's share of a weight stage is there (a pair's: the leader knows)
        auto arrive_w = [&](int s) {
            if (L::kPair)
                arrive_leader(full + s);
            else
                mbar_arrive(full + s);
        };
        bool ok = true;
        int g0 = 0, gk0 = 0, n = 0;  // steps and reduction steps before this tile
        int kjobs = 0;               // reduction steps of this group
        while (ok && it.next(tl)) {
            const int nk = tl.k_hi - tl.k_lo, steps = steps_of(tl);
            for (int i = (G - g0) & (kGroups - 1); ok && i < steps; i += kGroups) {
                // the weight stage is taken as late as possible: the codes
                // are read before the wait
                const int sw = (g0 + i) % L::kP;
                uint8_t* wst = smem + L::kOffW + sw * L::kWStage;
                // the stage's step before has been consumed; a stage's first step
                // has nothing to wait for (the phase before a barrier's first
                // counts as complete)
                const uint32_t w_par = static_cast<uint32_t>((g0 + i) / L::kP - 1) & 1u;
                if (i < nk) {
                    const int gk = gk0 + i, sc = gk % L::kPC;
                    ok = wait_both(c_full + 2 * G + (kjobs & 1), static_cast<uint32_t>(kjobs >> 1) & 1u, empty + sw,
                                   w_par, tmo, a.status);
                    if (!ok) break;
                    ++kjobs;
                    const uint32_t codes = smem_u32(smem + L::kOffC + sc * L::kCStage);
                    uint4 ca[kU], cb[kU];
                    uint32_t dst[kU], swz;
                    if (!kTransW) {
                        // rows t and t + 128 of the weight tile: 32 code bytes, 32-byte swizzle
                        const uint32_t s32 = (t >> 2) & 1;
                        swz = t & 7;
#pragma unroll
                        for (int u = 0; u < kU; ++u) {
                            const uint32_t crow = codes + (t + 128 * u) * 32;
                            ca[u] = lds128(crow + ((0 ^ s32) << 4));
                            cb[u] = lds128(crow + ((1 ^ s32) << 4));
                            dst[u] = smem_u32(wst) + (t + 128 * u) * 128 + (swz << 4);
                        }
                    } else {
                        // reduction row nl, k-blocks b and b + 2 of the tile's four
                        const uint32_t nl = t & 63, b = t >> 6;
                        const uint32_t crow = codes + nl * (L::kPair ? 64 : 128);
                        const uint32_t csw = L::kPair ? (nl >> 1) & 3 : nl & 7;  // 64- or 128-byte swizzle
                        swz = nl & 7;
#pragma unroll
                        for (int u = 0; u < kU; ++u) {
                            ca[u] = lds128(crow + (((2 * b + 4 * u) ^ csw) << 4));
                            cb[u] = lds128(crow + (((2 * b + 4 * u + 1) ^ csw) << 4));
                            dst[u] = smem_u32(wst) + (b + 2 * u) * 8192 + (nl >> 3) * 1024 + (nl & 7) * 128 + (swz << 4);
                        }
                    }
                    float cp[kU];
#pragma unroll
                    for (int u = 0; u < kU; ++u)
                        cp[u] = kNoDq ? raw_s[u] : __fmaf_rn(e4m3_to_f32(raw_q[u]), raw_s[u], mean);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(c_empty + sc);  // the codes have been read
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        const Nf4BlockLut lut = make_block_lut(tab.level, cp[u]);
                        const uint32_t words[8] = {ca[u].x, ca[u].y, ca[u].z, ca[u].w, cb[u].x, cb[u].y, cb[u].z, cb[u].w};
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            uint32_t o[4];
                            decode8(lut, words[j], o);
                            sts128(dst[u] ^ (static_cast<uint32_t>(j) << 4), o);  // rows are 128-byte aligned
                        }
                        if (u == 0) {  // the next step's constants, while this one's decoding goes on
                            pi += kGroups;
                            load_constants();
                        }
                    }
                    fence_proxy_async_smem();  // -> visible to the tensor core
                    __syncwarp();
                    if (lane == 0) arrive_w(sw);
                } else {
                    // rank-r step: B_e rows (forward) or A_e columns (dX) by TMA
                    pi += kGroups;
                    load_constants();
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(empty + sw, w_par, tmo, a.status));
                    if (!ok) break;
                    if (leader) {
                        if (crank == 0)
                            mbar_arrive_expect_tx(full + sw, L::kWStage * (L::kPair ? 2u : 1u));
                        else
                            arrive_w(sw);
                        for (int b = 0; b < (kTransW ? 2 * kU : 1); ++b) {
                            const int x = kTransW ? tl.w0 + w_off + 64 * b : 0, y = kTransW ? 0 : tl.w0 + w_off;
                            if (L::kPair)
                                tma_load_3d_pair(wst + b * 8192, &tm_lw, mapa_shared(smem_u32(full + sw), 0), x, y, tl.e);
                            else
                                tma_load_3d(wst + b * 8192, &tm_lw, full + sw, x, y, tl.e);
                        }
                    } else if (lane == 0) {
                        arrive_w(sw);
                    }
                    __syncwarp();
                }
            }
            g0 += steps;
            gk0 += nk;

            // ------------------------------------------------ epilogue --
            // (a warp whose wait ran out skips the work but meets the others
            // at the barriers; they leave together)
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(acc, static_cast<uint32_t>(n) & 1u, tmo, a.status)) && ok;
            tc_fence_after();
            const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16) + (CAP == 256 ? 0 : h * 256);
            // output column of this lane in the tile, and the first of this warp's
            // tokens: h is a half of a CTA's weight rows, the second UMMA of a
            // pair's 512 tokens, or every other 32 of a pair's 256
            const int nl = L::kPair ? w_off + q * 32 + lane : h * 128 + q * 32 + lane;
            const int tok0 = CAP == 512 ? 256 * h : 0;
            const int toks = CAP == 512 ? min(tl.rows - tok0, 256) : tl.rows;
            if (CAP != 64 || nk == KT) {
                // lane = output column, register = token: two neighbouring
                // lanes swap halves of a token pair, so each lane stores two
                // consecutive columns of one token and a warp instruction
                // covers two 64-byte row segments
                const int col = tl.w0 + (nl & ~1);
                const bool write = ok && col < a.out_cols;
                for (int c = CAP == 256 ? (2 * part + h) * 32 : part * 32; c < toks; c += CAP == 256 ? 128 : 64) {
                    uint32_t r[32];
                    tmem_ld32(trow + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const uint32_t give = (lane & 1) ? r[i] : r[i + 1];
                        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, give, 1);
                        const uint32_t lo = (lane & 1) ? got : r[i], hi = (lane & 1) ? r[i + 1] : got;
                        const int tok = c + i + (lane & 1);
                        if (write && tok < toks)
                            *reinterpret_cast<uint32_t*>(a.out + static_cast<int64_t>(tl.row0 + tok0 + tok) * a.out_cols + col) =
                                pack_bf16x2(__uint_as_float(lo), __uint_as_float(hi));
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
            } else if (CAP == 64) {
                // partial sums [token][256 columns] to this CTA's slot
                const int slot_floats = a.part_rows * 256;
                float* mine = a.part + ranges.slot(static_cast<int>(blockIdx.x), tl.id) * slot_floats + nl;
                for (int c = part * 32; c < tl.rows; c += 64) {
                    uint32_t r[32];
                    tmem_ld32(trow + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (ok && c + i < tl.rows) mine[(c + i) * 256] = __uint_as_float(r[i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(tmem_free);
                if (threadIdx.x == 0) pending->push(tl);
            }
            ++n;
            ok = all_ok(ok, kDeqWarps * 32);
        }
        // The tiles shared with other CTAs, once the loop (and the registers
        // it needs) is over: their last CTA to come here finishes them.
        if (CAP == 64 && pending->n > 0) {
            // the launch before this one has cleared the tickets
            asm volatile("griddepcontrol.wait;" ::: "memory");
            __threadfence();  // the parts are visible before the tickets
            ok = all_ok(ok, kDeqWarps * 32);
            if (threadIdx.x == 0) pending->take_tickets(ranges, a.tickets, ok);
            all_ok(true, kDeqWarps * 32);
            __threadfence();
            for (int k = 0; k < pending->n; ++k) {
                if (!pending->last[k]) continue;
                const Tile p = pending->tile[k];
                uint16_t* out = a.out + static_cast<int64_t>(p.row0) * a.out_cols + p.w0;
                const int c0 = ranges.first_cta(p.id);
                add_parts<float4>(a.part, a.part_rows * 256, ranges.slot(c0, p.id), c0, ranges.last_cta(p.id), p.rows,
                                  static_cast<int>(a.out_cols) - p.w0, static_cast<int>(threadIdx.x), kDeqWarps * 32,
                                  [&](int tok, int nc, const float4& v) {
                                      *reinterpret_cast<uint2*>(out + tok * a.out_cols + nc) =
                                          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                                  });
            }
        }
        if (!ok) {
            *abort_flag = 1;
            // a rank-r tile may still be landing in a weight stage
            if (leader)
                for (int j = max(0, g0 - 2 * L::kP); j < g0 + L::kP; ++j)
                    if ((j & (kGroups - 1)) == G)
                        mbar_wait(full + j % L::kP, static_cast<uint32_t>(j / L::kP) & 1u, tmo / 8, nullptr);
        }
        __syncwarp();
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
    // launched as a programmatic dependent, the grid completes only after its primary
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <bool kTransW, bool kNoDq, int CAP>
cudaError_t launch_one(const CUtensorMap& act, const CUtensorMap& codes, const CUtensorMap& lact, const CUtensorMap& lw,
                       const ExpertGemmArgs& a, const Nf4Tables& tab, cudaStream_t st) {
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
    return cudaLaunchKernelEx(&cfg, expert_gemm<kTransW, kNoDq, CAP>, act, codes, lact, lw, a, tab);
}

template <bool kTransW, int CAP>
cudaError_t launch_cap(const CUtensorMap& act, const CUtensorMap& codes, const CUtensorMap& lact, const CUtensorMap& lw,
                       const ExpertGemmArgs& a, const Nf4Tables& tab, cudaStream_t st) {
    return a.c.absmax ? launch_one<kTransW, true, CAP>(act, codes, lact, lw, a, tab, st)
                      : launch_one<kTransW, false, CAP>(act, codes, lact, lw, a, tab, st);
}

template <bool kTransW>
cudaError_t launch_dir(const CUtensorMap& act, const CUtensorMap& codes, const CUtensorMap& lact, const CUtensorMap& lw,
                       const ExpertGemmArgs& a, const Nf4Tables& tab, cudaStream_t st) {
    if (a.cap == 64) return launch_cap<kTransW, 64>(act, codes, lact, lw, a, tab, st);
    if (a.cap == 256) return launch_cap<kTransW, 256>(act, codes, lact, lw, a, tab, st);
    return launch_cap<kTransW, 512>(act, codes, lact, lw, a, tab, st);
}

template <bool kTransW, bool kNoDq, int CAP>
cudaError_t opt_in() {
    return cudaFuncSetAttribute(expert_gemm<kTransW, kNoDq, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(Lay<CAP>::kBytes));
}

template <int CAP>
cudaError_t opt_in_cap() {
    cudaError_t e;
    if ((e = opt_in<false, false, CAP>()) != cudaSuccess || (e = opt_in<false, true, CAP>()) != cudaSuccess ||
        (e = opt_in<true, false, CAP>()) != cudaSuccess)
        return e;
    return opt_in<true, true, CAP>();
}

}  // namespace

cudaError_t expert_gemm_init_device() {
    cudaError_t e;
    if ((e = opt_in_cap<64>()) != cudaSuccess || (e = opt_in_cap<256>()) != cudaSuccess) return e;
    return opt_in_cap<512>();
}

cudaError_t launch_expert_gemm(bool trans_w, const CUtensorMap& act, const CUtensorMap& codes, const CUtensorMap& lact,
                               const CUtensorMap& lw, const ExpertGemmArgs& a, const Nf4Tables& tab, cudaStream_t st) {
    if (a.E < 1 || a.E > kMaxExperts || a.ctas < 2 || (a.cap != 64 && a.cap != 256 && a.cap != 512) || a.rank_cols < 1 || a.rank_cols > 64)
        return cudaErrorInvalidValue;
    return trans_w ? launch_dir<true>(act, codes, lact, lw, a, tab, st)
                   : launch_dir<false>(act, codes, lact, lw, a, tab, st);
}

}  // namespace qlora
