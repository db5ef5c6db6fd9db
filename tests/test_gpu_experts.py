"""GPU parity of a layer of experts (rows grouped by expert, ragged) against
plain fp64 arithmetic on the oracle's dequantised weights.

Tolerances, per element, counted from the roundings:
  - a bf16 result is off by at most half a step, 2^-8 of its value;
  - the rank-r input enters Y and dX as its bf16 rounding: 2^-8 of |sT| |B|;
  - the tensor core adds 16 products at a time into an fp32 accumulator that
    loses at most one unit, 2^-23 of the running sum, per addition; the running
    sum is at most the sum of magnitudes S, so n terms lose (n / 16 + c) 2^-23 S
    (c = 64 covers the rank-r step, the fp32 additions between parts and the
    operands' own 2^-16 .. 2^-24 splits where S carries them).
"""
import numpy as np
import pytest
import torch

import oracle
import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_09_b200 import build
    build.build()
    import bit_nf4_quantized_09_b200 as q
    assert torch.cuda.is_available()
    return q


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def acc(n):
    return (n / 16 + 64) * U


def within(name, got, ref, tol):
    bad = np.abs(got - ref) > tol
    worst = np.max(np.abs(got - ref) / np.maximum(tol, 1e-300)) if got.size else 0.0
    print(f"{name}: worst error / tolerance = {worst:.3f}")
    assert np.array_equal(np.isfinite(got), np.isfinite(ref)), name
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:3].tolist())


def what_of(W, dq):
    if dq:
        z = oracle.quantize_nf4(W.numpy())
        bits = oracle.dequant_bf16_bits(z["codes"], z["qabsmax"], z["s2"], z["mean"], z["N"], z["K"])
    else:
        z = oracle.quantize_nf4_nodq(W.numpy())
        bits = oracle.dequant_bf16_bits_nodq(z["codes"], z["absmax"], z["N"], z["K"])
    return oracle.bf16_bits_to_f64(bits)


def case(counts, N, K, r, dq=True, lead=0, pad=0, seed=700):
    """Inputs of a layer of len(counts) experts; `lead` rows before the first
    expert's and `pad` behind the last one's belong to nobody."""
    E, M = len(counts), lead + sum(counts) + pad
    cfg = synth.custom(N=E * N, K=K, M=M, r=r, seed_base=seed)
    g = torch.Generator().manual_seed(seed)
    return dict(E=E, N=N, K=K, M=M, r=r, dq=dq, alpha=cfg.alpha, W=synth.weight(cfg), X=synth.activations(cfg),
                A=torch.randn(E * r, K, generator=g).mul_(K ** -0.5).bfloat16(),
                B=torch.randn(E * N, r, generator=g).mul_(0.1).bfloat16(),
                dY=torch.randn(M, N, generator=g).bfloat16(),
                off=np.concatenate([[0], np.cumsum(counts)]) + lead)


def quantised(q, t):
    return (q.quantize_nf4 if t["dq"] else q.quantize_nf4_nodq)(t["W"].cuda())


def run(q, t, sT_given=True):
    w = quantised(q, t)
    X, A, B, dY = (t[k].cuda() for k in ("X", "A", "B", "dY"))
    off = torch.tensor(t["off"], dtype=torch.int32, device="cuda")
    Y = torch.full((t["M"], t["N"]), 7.0, dtype=torch.bfloat16, device="cuda")
    sT = torch.full((t["M"], 2 * t["r"]), 7.0, dtype=torch.bfloat16, device="cuda")
    dX = torch.full((t["M"], t["K"]), 7.0, dtype=torch.bfloat16, device="cuda")
    q.linear_fwd_experts(X, w, A, B, off, t["E"], t["alpha"], Y=Y, sT=sT)
    _, dA, dB = q.linear_bwd_experts(dY, X, w, A, B, off, t["E"], t["alpha"], sT=sT if sT_given else None, dX=dX)
    torch.cuda.synchronize()
    return dict(Y=Y, sT=sT, dX=dX, dA=dA, dB=dB)


def compare(t, g, off=None):
    off = t["off"] if off is None else off
    What = what_of(t["W"], t["dq"])
    E, N, K, r, s = t["E"], t["N"], t["K"], t["r"], t["alpha"] / t["r"]
    free = np.ones(t["M"], bool)
    for e in range(E):
        m = slice(off[e], off[e + 1])
        free[m] = False
        We, A, B = What[e * N:(e + 1) * N], f64(t["A"][e * r:(e + 1) * r]), f64(t["B"][e * N:(e + 1) * N])
        X, dY = f64(t["X"][m]), f64(t["dY"][m])
        sT, sTa = s * X @ A.T, s * np.abs(X) @ np.abs(A).T
        sU, sUa = s * dY @ B, s * np.abs(dY) @ np.abs(B)
        got_T = f64(g["sT"][m])
        got_T = got_T[:, :r] + got_T[:, r:]
        within(f"sT[{e}]", got_T, sT, 2.0 ** -16 * np.abs(sT) + acc(K) * sTa)
        Y = X @ We.T + sT @ B.T
        within(f"Y[{e}]", f64(g["Y"][m]), Y, 2.0 ** -8 * np.abs(Y) + (2.0 ** -8 + acc(r)) * np.abs(sT) @ np.abs(B).T
               + acc(K) * (np.abs(X) @ np.abs(We).T + sTa @ np.abs(B).T))
        dX = dY @ We + sU @ A
        within(f"dX[{e}]", f64(g["dX"][m]), dX, 2.0 ** -8 * np.abs(dX) + (2.0 ** -8 + acc(r)) * np.abs(sU) @ np.abs(A)
               + acc(N) * (np.abs(dY) @ np.abs(We) + sUa @ np.abs(A)))
        n = max(len(X), 1)
        dA, dB = sU.T @ X, dY.T @ got_T
        within(f"dA[{e}]", f64(g["dA"][e * r:(e + 1) * r]), dA, acc(n) * np.abs(sU).T @ np.abs(X) + acc(N) * sUa.T @ np.abs(X))
        within(f"dB[{e}]", f64(g["dB"][e * N:(e + 1) * N]), dB, acc(n) * np.abs(dY).T @ np.abs(got_T))
        if len(X):
            # read-outs every 512 rows and three-term operands: far below one
            # bf16 rounding, 2^-8, of the rank-r input
            for name, got, ref in (("dA", f64(g["dA"][e * r:(e + 1) * r]), dA), ("dB", f64(g["dB"][e * N:(e + 1) * N]), dB)):
                assert np.linalg.norm(got - ref) <= 1e-5 * np.linalg.norm(ref), (name, e)
    for k in ("Y", "sT", "dX"):
        assert torch.all(g[k].cpu()[torch.from_numpy(free)] == 7.0), k  # rows of nobody


CASES = {
    # few tokens, reduction split over clusters
    "one_row": dict(counts=[0, 1, 0], N=512, K=512, r=8),
    "single_tokens": dict(counts=[1, 1, 0, 1], N=264, K=1088, r=16),
    "decode": dict(counts=[5, 0, 17, 3, 8, 16, 1, 14], N=520, K=640, r=32),
    "decode_64": dict(counts=[64, 33], N=1024, K=2048, r=64),
    "few_long_experts": dict(counts=[200, 130], N=264, K=320, r=64),
    # token tiles of 64 without and with ragged ends, narrow and wide
    "ragged_small": dict(counts=[65, 0, 127, 1, 64], N=776, K=320, r=16, pad=9),
    "tiny_shapes": dict(counts=[3, 2], N=8, K=64, r=8),
    # tiles of up to 256 tokens
    "ragged_big": dict(counts=[257, 300, 0, 511, 256, 90], N=7688, K=192, r=16, lead=5, pad=37),
    "dx_big": dict(counts=[290, 77, 400], N=200, K=12800, r=32, pad=3),
    "no_double_quant": dict(counts=[40, 100, 7], N=520, K=576, r=8, dq=False),
    "no_double_quant_odd_blocks": dict(counts=[300, 280], N=19208, K=320, r=64, dq=False),
    "long_expert": dict(counts=[3000, 60], N=136, K=128, r=64),
}


@pytest.mark.parametrize("name", CASES)
def test_experts_against_fp64(q, name):
    t = case(**CASES[name])
    compare(t, run(q, t))


# forwards in tiles of 8 and 16 rows: constants in whole words and not, one
# expert with far more rows than the mean, tiles shared among CTAs beside whole
# ones, a reduction that ends inside a step
FEW = {
    "tiles_of_8": dict(counts=[1, 0, 2, 6], N=520, K=256, r=8, dq=False, lead=3, pad=2),
    "tiles_of_16": dict(counts=[9, 16, 0, 7], N=264, K=320, r=16, dq=False),
    "words_16": dict(counts=[2, 11, 4], N=72, K=4096, r=64, lead=3, pad=5),
    "skewed": dict(counts=[0, 60, 0, 0, 0, 4, 0, 0], N=264, K=1088, r=32),
    "whole_and_shared": dict(counts=[1 + i % 4 for i in range(80)], N=264, K=1600, r=8),
}


@pytest.mark.parametrize("name", FEW)
def test_few_rows_against_fp64(q, name):
    t = case(**FEW[name])
    a = run(q, t)
    compare(t, a)
    b = run(q, t)
    for k in a:
        assert torch.equal(a[k], b[k]), k


# tiles of 256 and 512 tokens on pairs of CTAs: token counts around the tiles'
# sizes and the 32-row granularity, weight tiles of which one CTA has no row
PAIRS = {
    "edges_512": dict(counts=[512, 513, 31, 1, 257, 289], N=2440, K=448, r=16),
    "edges_256": dict(counts=[33, 200, 64, 128, 97], N=264, K=1088, r=8, dq=False, lead=1),
    "one_half": dict(counts=[130, 70], N=2056, K=2112, r=64, pad=3),
    "many_rounds": dict(counts=[100] * 40, N=904, K=64, r=32),
}


@pytest.mark.parametrize("name", PAIRS)
def test_pairs_against_fp64(q, name):
    t = case(**PAIRS[name])
    a = run(q, t)
    compare(t, a)
    b = run(q, t)
    for k in a:
        assert torch.equal(a[k], b[k]), k


# every instantiation of the matmul, by the tile rows that the sizes choose for the
# forward and for dX: both storages, tiles of 64 whole, shared out and both in one call
TILES = {
    "64_shared": (64, 256, dict(counts=[33, 64, 17], N=264, K=960, r=16)),
    "64_shared_fp32": (64, 256, dict(counts=[33, 64, 17], N=264, K=960, r=8, dq=False, lead=2)),
    "64_whole_and_shared": (64, 64, dict(counts=[14] * 60 + [1, 27] * 8, N=264, K=1088, r=16)),
    "64_whole_and_shared_fp32": (64, 64, dict(counts=[14] * 60 + [1, 27] * 8, N=264, K=1088, r=32, dq=False)),
    "512_and_64_shared": (512, 64, dict(counts=[200, 100, 350, 1], N=8008, K=1024, r=8)),
    "512_and_64_shared_fp32": (512, 64, dict(counts=[200, 100, 350, 1], N=8008, K=1024, r=64, dq=False)),
    "64_and_512": (64, 512, dict(counts=[600, 290, 31], N=520, K=20032, r=16, pad=2)),
    "64_and_512_fp32": (64, 512, dict(counts=[600, 290, 31], N=520, K=20032, r=32, dq=False)),
    "512_both": (512, 512, dict(counts=[513, 300, 257, 1, 0, 1024, 512, 290, 31], N=1032, K=1088, r=64)),
    # forwards of few rows behind each of the two down-projections
    "16_tensor_down": (16, 64, dict(counts=[8, 0, 11, 7, 30, 1, 6, 3], N=72, K=11008, r=64)),
    "8_tensor_down": (8, 64, dict(counts=[5] * 12, N=40, K=11008, r=64, lead=1, pad=2)),
    "16_core_down": (16, 64, dict(counts=[8, 0, 11, 7, 30, 1, 6, 3], N=72, K=4096, r=64)),
    "256_both": (256, 256, dict(counts=[600, 290, 31], N=2440, K=2112, r=8)),
    "256_both_fp32": (256, 256, dict(counts=[600, 290, 31], N=2440, K=2112, r=16, dq=False)),
}


@pytest.mark.parametrize("name", TILES)
def test_tiles_against_fp64(q, name):
    fwd, dx, sizes = TILES[name]
    t = case(**sizes)
    assert q.tile_rows_experts(q.OP_FWD, t["M"], t["N"], t["K"], t["E"]) == fwd
    assert q.tile_rows_experts(q.OP_BWD, t["M"], t["N"], t["K"], t["E"]) == dx
    a = run(q, t)
    compare(t, a)
    b = run(q, t)
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("counts,N,K,r", [([5, 2], 136, 64, 8), ([40, 30], 264, 128, 16), ([300, 200], 520, 960, 32),
                                          ([700, 513], 392, 64, 64), ([3, 9], 264, 2048, 64)])
def test_rank_r_terms_are_not_rounded_away(q, counts, N, K, r):
    """On short reductions, and in the forward of few rows, sT and sU enter Y and
    dX as two bf16 terms: what they leave is 2^-8 of 2^-8 of them."""
    t = case(counts, N=N, K=K, r=r)
    g = run(q, t)
    What = what_of(t["W"], True)
    s = t["alpha"] / r
    for e in range(t["E"]):
        m = slice(t["off"][e], t["off"][e + 1])
        We, A, B = What[e * N:(e + 1) * N], f64(t["A"][e * r:(e + 1) * r]), f64(t["B"][e * N:(e + 1) * N])
        X, dY = f64(t["X"][m]), f64(t["dY"][m])
        sT, sTa = s * X @ A.T, s * np.abs(X) @ np.abs(A).T
        Y = X @ We.T + sT @ B.T
        within("Y", f64(g["Y"][m]), Y, 2.0 ** -8 * np.abs(Y) + (2.0 ** -16 + acc(r)) * np.abs(sT) @ np.abs(B).T
               + acc(K) * (np.abs(X) @ np.abs(We).T + sTa @ np.abs(B).T))
        if N < 1024:
            sU, sUa = s * dY @ B, s * np.abs(dY) @ np.abs(B)
            dX = dY @ We + sU @ A
            within("dX", f64(g["dX"][m]), dX, 2.0 ** -8 * np.abs(dX) + (2.0 ** -16 + acc(r)) * np.abs(sU) @ np.abs(A)
                   + acc(N) * (np.abs(dY) @ np.abs(We) + sUa @ np.abs(A)))


@pytest.mark.parametrize("counts,N,K,r", [([20, 20], 1096, 2048, 8), ([130, 77], 1024, 1024, 32),
                                          ([300, 200] * 8, 1032, 1088, 64), ([5, 2], 1024, 1024, 16)])
def test_strong_adapter_on_long_reductions(q, counts, N, K, r):
    """sT and sU are 257 and 256 times a power of two by turns (257 does not fit
    bf16's 8 bits), the adapter's other factor cancels all but their difference,
    the base weight is zero: every product and sum is exact, and so is the result
    where two terms of sT and sU reach Y and dX; one term gives zeros."""
    E, M = len(counts), sum(counts)
    g = torch.Generator().manual_seed(r)
    ones = lambda n: torch.stack([torch.randperm(n, generator=g) < 257 - j % 2 for j in range(E * r)]).float()  # noqa: E731
    power = lambda n: torch.tensor([1.0, -2.0, 0.5, 4.0])[torch.randint(4, (n,), generator=g)]  # noqa: E731
    sign = torch.tensor([1.0, -1.0] * (r // 2))
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    w = q.quantize_nf4(torch.zeros(E * N, K, device="cuda"))
    expert = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))
    bf = lambda t: t.bfloat16().cuda()  # noqa: E731
    # Y[m, n] = x[m] b[n] (257 - 256) r / 2
    x, b = power(M), power(E * N)
    Y, sT = q.linear_fwd_experts(bf(x[:, None].expand(M, K)), w, bf(ones(K)), bf(b[:, None] * sign), off, E, float(r))
    t = sT.float().cpu()
    assert torch.equal(t[:, :r] + t[:, r:], x[:, None] * (256.5 + 0.5 * sign))
    assert torch.equal(Y.float().cpu(), x[:, None] * b.reshape(E, N)[expert] * (r / 2))
    # dX[m, k] = y[m] a[k] (257 - 256) r / 2
    y, a = power(M), power(E * K).reshape(E, K)
    B = ones(N).reshape(E, r, N).transpose(1, 2).reshape(E * N, r)
    A = (sign[None, :, None] * a[:, None, :]).reshape(E * r, K)
    dX, _, _ = q.linear_bwd_experts(bf(y[:, None].expand(M, N)), bf(torch.zeros(M, K)), w, bf(A), bf(B), off, E, float(r))
    assert torch.equal(dX.float().cpu(), y[:, None] * a[expert] * (r / 2))


@pytest.mark.parametrize("counts", [[3, 5, 1], [9, 14, 6]], ids=["8", "16"])
def test_few_rows_do_not_leak(q, counts):
    """As for many rows: NaN and infinities stay in their own rows."""
    t = case(counts, N=264, K=320, r=16, lead=2, pad=4)
    clean = run(q, t)["Y"].cpu()
    dirty = dict(t, X=t["X"].clone())
    dirty["X"][:2], dirty["X"][-4:], dirty["X"][t["off"][1] + 1] = float("nan"), float("inf"), float("nan")
    got = run(q, dirty)["Y"].cpu()
    mine = torch.zeros(t["M"], dtype=torch.bool)
    mine[t["off"][1] + 1] = True
    assert torch.equal(clean[~mine], got[~mine])
    assert torch.isnan(got[mine].float()).all()


def test_recomputed_rank_input_and_determinism(q):
    t = case([70, 200, 0, 33], N=264, K=448, r=32)
    a, b, c = run(q, t), run(q, t), run(q, t, sT_given=False)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    for k in ("dX", "dA", "dB"):
        assert torch.equal(a[k], c[k]), k


@pytest.mark.parametrize("counts", [[9, 30, 12], [100, 70, 300]], ids=["split", "tiles"])
def test_one_expert_equals_a_layer_of_its_own(q, counts):
    """Each expert's rows give what a call with that expert alone gives."""
    t = case(counts, N=264, K=320, r=16)
    g = run(q, t)
    w = quantised(q, t)
    What = what_of(t["W"], True)
    for e in range(t["E"]):
        m = slice(t["off"][e], t["off"][e + 1])
        off = torch.tensor([0] * (e + 1) + [counts[e]] * (t["E"] - e), dtype=torch.int32, device="cuda")
        Y, sT = q.linear_fwd_experts(t["X"][m].cuda(), w, t["A"].cuda(), t["B"].cuda(), off, t["E"], t["alpha"])
        torch.cuda.synchronize()
        # another batch may split the reduction another way, and round sT the
        # other way: each result is off by half a bf16 step of its own, by the
        # accumulation errors, and by sT's rounding, 2^-8 of |sT| |B|
        A, B = f64(t["A"][e * t["r"]:(e + 1) * t["r"]]), f64(t["B"][e * t["N"]:(e + 1) * t["N"]])
        X = f64(t["X"][m])
        sT_, sTa = t["alpha"] / t["r"] * X @ A.T, t["alpha"] / t["r"] * np.abs(X) @ np.abs(A).T
        size = np.abs(X) @ np.abs(What[e * t["N"]:(e + 1) * t["N"]]).T + sTa @ np.abs(B).T
        y, s = f64(g["Y"][m]), f64(g["sT"][m])
        within("Y", f64(Y), y, 2 * (2.0 ** -8 * np.abs(y) + 2.0 ** -8 * np.abs(sT_) @ np.abs(B).T + acc(t["K"]) * size))
        r = t["r"]
        within("sT", f64(sT)[:, :r] + f64(sT)[:, r:], s[:, :r] + s[:, r:],
               2 * (2.0 ** -16 * np.abs(sT_) + acc(t["K"]) * sTa))


def test_rows_of_nobody_and_of_other_experts_do_not_leak(q):
    """NaN and infinities in rows of no expert reach nothing, and those in one
    expert's rows stay in its own rows and gradients."""
    t = case([70, 33, 65], N=264, K=320, r=16, lead=2, pad=20)
    clean = run(q, t)
    dirty = dict(t, X=t["X"].clone(), dY=t["dY"].clone())
    dirty["X"][:2], dirty["X"][-20:] = float("nan"), float("inf")
    dirty["dY"][:2], dirty["dY"][-20:] = float("inf"), float("nan")
    got = run(q, dirty)
    for k in clean:
        assert torch.equal(clean[k], got[k]), k
    hot = dict(t, X=t["X"].clone(), dY=t["dY"].clone())
    hot["X"][t["off"][1] + 4] = float("nan")       # one row of expert 1
    hot["dY"][t["off"][1] + 4] = float("inf")
    got = run(q, hot)
    N, r = t["N"], t["r"]
    mine = torch.zeros(t["M"], dtype=torch.bool)
    mine[t["off"][1] + 4] = True
    for k in ("Y", "dX", "sT"):
        assert torch.equal(clean[k].cpu()[~mine], got[k].cpu()[~mine]), k
        assert not torch.isfinite(got[k].cpu()[mine].float()).any() if k != "sT" else True
    for k, n in (("dA", r), ("dB", N)):
        for e in (0, 2):
            assert torch.equal(clean[k][e * n:(e + 1) * n], got[k][e * n:(e + 1) * n]), (k, e)
        assert not torch.isfinite(got[k][n:2 * n]).any(), k


def test_empty_batches_and_experts(q):
    t = case([0, 0, 0], N=64, K=64, r=8, pad=5)
    g = run(q, t)
    assert torch.count_nonzero(g["dA"]) == 0 and torch.count_nonzero(g["dB"]) == 0
    for k in ("Y", "sT", "dX"):
        assert torch.all(g[k] == 7.0)
    t = case([0, 0], N=64, K=64, r=8)
    g = run(q, t)                                   # M == 0
    assert g["Y"].shape == (0, 64)
    assert torch.count_nonzero(g["dA"]) == 0 and torch.count_nonzero(g["dB"]) == 0


@pytest.mark.parametrize("raw", [[0, 50, 30, 90], [-5, 20, 20, 1000], [70, 70, 70, 70], [10, 5, 2, 1]])
def test_offsets_are_made_safe(q, raw):
    """Offsets that decrease or leave [0, M] act as their running maximum,
    clamped."""
    t = case([30, 30, 30], N=72, K=128, r=8)
    safe = np.maximum.accumulate(np.clip(raw, 0, t["M"]))
    t["off"] = np.array(raw)
    compare(t, run(q, t), off=safe)


def test_many_experts(q):
    rng = np.random.default_rng(3)
    counts = rng.integers(0, 4, 512)
    t = case(counts.tolist(), N=8, K=64, r=8)
    compare(t, run(q, t))


def test_gradients_against_differences(q):
    """<dY, Y(X + d)> - <dY, Y(X - d)> against <dX, 2 d>, and the same for A and
    B: Y is linear in each, so the differences are exact up to the roundings,
    2^-8 of each product's terms."""
    t = case([20, 45], N=128, K=128, r=16)
    w = quantised(q, t)
    off = torch.tensor(t["off"], dtype=torch.int32, device="cuda")
    X, A, B, dY = (t[k].cuda() for k in ("X", "A", "B", "dY"))
    gen = torch.Generator(device="cuda").manual_seed(1)

    def value(X, A, B):
        Y, _ = q.linear_fwd_experts(X, w, A, B, off, t["E"], t["alpha"])
        return (Y.double() * dY.double())

    _, sT = q.linear_fwd_experts(X, w, A, B, off, t["E"], t["alpha"])
    dX, dA, dB = q.linear_bwd_experts(dY, X, w, A, B, off, t["E"], t["alpha"], sT=sT)
    for name, base, grad in (("X", X, dX), ("A", A, dA), ("B", B, dB)):
        d = torch.randn(base.shape, generator=gen, device="cuda") * base.float().abs().mean()
        up, down = (base.float() + d).bfloat16(), (base.float() - d).bfloat16()
        args = lambda v: [v if name == k else o for k, o in (("X", X), ("A", A), ("B", B))]  # noqa: E731
        p, m = value(*args(up)), value(*args(down))
        got = (p.sum() - m.sum()).item()
        ref = (grad.double() * (up.double() - down.double())).sum().item()
        # independent roundings of every output, and of dX or of sT
        tol = 4 * 2.0 ** -8 * (p.square().sum() + m.square().sum()).sqrt().item() + \
            4 * 2.0 ** -8 * (grad.double() * (up.double() - down.double())).square().sum().sqrt().item()
        print(name, got, ref, tol)
        assert abs(got - ref) <= tol, name


def test_other_stream_and_captured_replay(q):
    """A call on another stream and a captured graph replayed on new inputs
    give the eager bits."""
    t = case([40, 300, 0, 9], N=264, K=320, r=16)
    w = quantised(q, t)
    off = torch.tensor(t["off"], dtype=torch.int32, device="cuda")
    X, A, B, dY = (t[k].cuda() for k in ("X", "A", "B", "dY"))
    E, al = t["E"], t["alpha"]
    q.set_check_device_status(False)

    def step(ws=None, wsb=None):
        Y, sT = q.linear_fwd_experts(X, w, A, B, off, E, al, ws=ws)
        return (Y, sT) + q.linear_bwd_experts(dY, X, w, A, B, off, E, al, sT=sT, ws=wsb)

    ref = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(ref, other):
        assert torch.equal(a, b)
    ws = torch.empty(q.workspace_bytes_experts(q.OP_FWD, t["M"], t["N"], t["K"], t["r"], E), dtype=torch.uint8, device="cuda")
    wsb = torch.empty(q.workspace_bytes_experts(q.OP_BWD, t["M"], t["N"], t["K"], t["r"], E), dtype=torch.uint8,
                      device="cuda")
    with torch.cuda.stream(s):
        step(ws, wsb)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(ws, wsb)
    X.copy_(X.flip(0))
    off.copy_(torch.tensor([0, 100, 100, 340, 349], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    new = step()
    for a, b in zip(out, new):
        assert torch.equal(a, b)
    assert q.device_status(ws) == 0 and q.device_status(wsb) == 0


@pytest.mark.parametrize("counts", [[1, 0, 2], [30, 45, 20], [300, 40, 513]], ids=["few", "small", "pairs"])
def test_two_streams_at_once(q, counts):
    """Two streams run forwards and backwards of different batches at the same
    time, each with workspaces of its own."""
    ts = [case(counts, N=1032, K=2048, r=16, seed=s) for s in (71, 72)]
    ref = [run(q, t) for t in ts]
    q.set_check_device_status(False)
    state = []
    for t in ts:
        off = torch.tensor(t["off"], dtype=torch.int32, device="cuda")
        ws = [torch.empty(q.workspace_bytes_experts(op, t["M"], t["N"], t["K"], t["r"], t["E"]), dtype=torch.uint8,
                          device="cuda") for op in (q.OP_FWD, q.OP_BWD)]
        state.append((quantised(q, t), [t[k].cuda() for k in ("X", "A", "B", "dY")], off, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    out = [[], []]
    for _ in range(4):
        for i, (w, (X, A, B, dY), off, ws, s) in enumerate(state):
            with torch.cuda.stream(s):
                Y, sT = q.linear_fwd_experts(X, w, A, B, off, ts[i]["E"], ts[i]["alpha"], ws=ws[0])
                dX, dA, dB = q.linear_bwd_experts(dY, X, w, A, B, off, ts[i]["E"], ts[i]["alpha"], sT=sT, ws=ws[1])
                out[i].append(dict(Y=Y, sT=sT, dX=dX, dA=dA, dB=dB))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(q.device_status(x) == 0 for x in state[i][3])
        for got in out[i]:
            for k in got:
                assert torch.equal(got[k], ref[i][k]), (i, k)


def test_graphs_that_share_a_workspace(q):
    """Two graphs captured with one workspace, replayed in turn on one stream; the
    workspace is the larger batch's."""
    ts = [case([300, 0, 513], N=264, K=448, r=16, seed=81), case([2, 1, 0], N=264, K=448, r=16, seed=82)]
    ref = [run(q, t) for t in ts]
    q.set_check_device_status(False)
    n = max(q.workspace_bytes_experts(op, ts[0]["M"], 264, 448, 16, 3) for op in (q.OP_FWD, q.OP_BWD))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, outs, keep = [], [], []
    for t in ts:
        w, off = quantised(q, t), torch.tensor(t["off"], dtype=torch.int32, device="cuda")
        X, A, B, dY = (t[k].cuda() for k in ("X", "A", "B", "dY"))
        keep.append((w, off, X, A, B, dY))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            Y, sT = q.linear_fwd_experts(X, w, A, B, off, 3, t["alpha"], ws=ws)
            dX, dA, dB = q.linear_bwd_experts(dY, X, w, A, B, off, 3, t["alpha"], sT=sT, ws=ws)
        graphs.append(g)
        outs.append(dict(Y=Y, sT=sT, dX=dX, dA=dA, dB=dB))
    for _ in range(2):
        for i in range(2):
            for v in outs[i].values():
                v.zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert q.device_status(ws) == 0
            for k, v in outs[i].items():
                assert torch.equal(v, ref[i][k]), (i, k)


# ------------------------------------------------------------------- order --

def order_ref(ids, E):
    key = [v if 0 <= v < E else E for v in ids]
    order = sorted(range(len(ids)), key=lambda m: key[m])
    return order, [sum(k < e for k in key) for e in range(E + 1)]


@pytest.mark.parametrize("M,E", [(0, 4), (1, 1), (2, 8), (31, 3), (33, 512), (1000, 7), (1024, 32), (5000, 512),
                                 (9001, 33)])
def test_order(q, M, E):
    g = torch.Generator().manual_seed(M + E)
    ids = torch.randint(-2, E + 2, (M,), generator=g, dtype=torch.int32)
    order, offsets = q.expert_order(ids.cuda(), E)
    torch.cuda.synchronize()
    ro, rf = order_ref(ids.tolist(), E)
    assert order.tolist() == ro
    assert offsets.tolist() == rf


@pytest.mark.parametrize("M,E", [(4097, 512), (65536, 64), (65537, 3), (150001, 20)])
def test_order_of_long_batches(q, M, E):
    """Pieces of up to 256 rows per warp, and longer ones."""
    g = torch.Generator().manual_seed(M)
    ids = torch.randint(-1, E + 1, (M,), generator=g, dtype=torch.int32)
    order, offsets = q.expert_order(ids.cuda(), E)
    torch.cuda.synchronize()
    key = torch.where((ids >= 0) & (ids < E), ids, torch.full_like(ids, E)).long()
    assert torch.equal(order.cpu().long(), torch.sort(key, stable=True).indices)
    assert offsets.tolist() == [int((key < e).sum()) for e in range(E + 1)]


def test_order_of_one_expert_and_none(q):
    for v in (0, 2, -1):
        ids = torch.full((777,), v, dtype=torch.int32, device="cuda")
        order, offsets = q.expert_order(ids, 3)
        torch.cuda.synchronize()
        assert order.tolist() == list(range(777))
        assert offsets.tolist() == [777 if 0 <= v < e else 0 for e in range(4)]
