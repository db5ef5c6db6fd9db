"""GPU parity of the 8-bit integer quantiser and product.

Codes, scales and outputs are compared bit for bit: the codes are the exactly
rounded quotients (127 x exactly, one division: fp64 separates every quotient
from a half, which are at least 2^-32 apart), the integer sums are exact, and
the result is three fp32 roundings and one to bf16 in a stated order."""
import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_09_b200 import build
    build.build()
    import bit_nf4_quantized_09_b200 as q
    assert torch.cuda.is_available()
    return q


def quantised(x):
    """(codes, scale) of the rows of a CPU tensor, from the definition."""
    x = x.double()
    a = x.abs().amax(1, keepdim=True)
    codes = torch.where(a > 0, torch.round(127 * x / torch.where(a > 0, a, torch.ones_like(a))), torch.zeros_like(x))
    return codes.to(torch.int8), (a[:, 0].float() / 127)


def product(x, codes, scale):
    """Y from the definition: exact sums, then the kernel's roundings."""
    qx, xs = quantised(x)
    s = qx.double() @ codes.double().t()
    return (s.float() * (xs[:, None] * scale[None, :])).bfloat16()


def rows(M, K, seed, dtype=torch.bfloat16, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, K, generator=g) * std).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,K", [(1, 16), (8, 64), (33, 2048), (7, 8192), (5, 8208), (3, 40000), (300, 4096)])
def test_quantise_rows_bit_exact(q, N, K, dtype):
    x = rows(N, K, N + K, dtype, 0.02)
    w = q.quantize_int8(x.cuda())
    torch.cuda.synchronize()
    codes, scale = quantised(x)
    assert torch.equal(w.codes.cpu(), codes)
    assert torch.equal(w.scale.cpu(), scale)


def test_quantise_ties_and_extremes(q):
    """Halves go to the even code; rows of zeros, tiny and huge rows."""
    K = 256
    k = torch.arange(K, dtype=torch.float32)
    tie = (k - 127.5).clamp(-127, 127)          # a = 127: every quotient is a half
    tie[0] = 127
    rowsx = [tie, tie * 2.0 ** -10, torch.zeros(K), tie * 2.0 ** -140, torch.full((K,), 2.0 ** -149),
             tie * 2.0 ** 120, -tie, torch.eye(1, K)[0] * 3e38, torch.full((K,), -1.0)]
    # quotients next to a half on either side
    a = torch.tensor(1.9999999, dtype=torch.float32)
    near = ((k % 127).double() + 0.5) * a.double() / 127
    near[0] = a
    rowsx += [near.float(), torch.nextafter(near.float(), torch.zeros(())).clamp(-a, a),
              torch.nextafter(near.float(), torch.full((), 9.0)).clamp(-a, a)]
    x = torch.stack(rowsx)
    w = q.quantize_int8(x.cuda())
    torch.cuda.synchronize()
    codes, scale = quantised(x)
    assert torch.equal(w.codes.cpu(), codes)
    assert torch.equal(w.scale.cpu(), scale)


def test_rows_that_are_not_finite(q):
    x = rows(6, 512, 5)
    x[1, 7], x[3, 500], x[4, 0] = float("nan"), float("inf"), float("-inf")
    bad = torch.tensor([1, 3, 4])
    good = torch.tensor([0, 2, 5])
    w = q.quantize_int8(x.cuda())
    c, s = w.codes.cpu(), w.scale.cpu()
    assert torch.isnan(s[bad]).all() and torch.count_nonzero(c[bad]) == 0
    codes, scale = quantised(x[good])
    assert torch.equal(c[good], codes) and torch.equal(s[good], scale)
    # as tokens: NaN rows of Y, no other row touched
    W = rows(264, 512, 6, torch.float32, 0.02)
    w8 = q.quantize_int8(W.cuda())
    Y = q.linear_int8(x.cuda(), w8).cpu()
    assert torch.isnan(Y[bad].float()).all()
    assert torch.equal(Y[good], product(x[good], *quantised(W)))


@pytest.mark.parametrize("M,N,K", [
    (1, 8, 16), (1, 520, 4096), (3, 264, 112), (16, 1024, 2048), (17, 1000, 640), (64, 2048, 1024), (65, 776, 320),
    (200, 4096, 528), (300, 40000, 144), (1000, 12808, 256), (257, 520, 131072 // 8)])
def test_product_bit_exact(q, M, N, K):
    X, W = rows(M, K, M + 1), rows(N, K, N + 2, torch.float32, 0.02)
    X[:, ::7] *= 8                        # outlier channels
    w = q.quantize_int8(W.cuda())
    Y = q.linear_int8(X.cuda(), w)
    torch.cuda.synchronize()
    assert torch.equal(Y.cpu(), product(X, *quantised(W)))


def test_longest_reduction_does_not_overflow(q):
    """Every product at its largest: 127 * 127 * 131072 < 2^31."""
    K = 131072
    X, W = torch.ones(2, K).bfloat16(), torch.ones(8, K)
    W[1] = -1
    Y = q.linear_int8(X.cuda(), q.quantize_int8(W.cuda()))
    assert torch.equal(Y.cpu(), product(X, *quantised(W)))


@pytest.mark.parametrize("counts,N,K,lead,pad", [
    ([1, 0, 1], 264, 512, 0, 0), ([5, 16, 0, 43], 520, 640, 0, 3), ([64, 64], 1024, 2048, 0, 0),
    ([300, 0, 257, 511, 90], 10248, 144, 7, 33), ([100, 1, 70], 776, 336, 1, 0)])
def test_experts_bit_exact(q, counts, N, K, lead, pad):
    E, M = len(counts), lead + sum(counts) + pad
    X, W = rows(M, K, M), rows(E * N, K, N, torch.float32, 0.02)
    X[:lead], X[M - pad:] = float("nan"), float("nan")     # rows of nobody
    off = np.concatenate([[0], np.cumsum(counts)]) + lead
    w = q.quantize_int8(W.cuda())
    Y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    q.linear_int8_experts(X.cuda(), w, offsets, E, Y=Y)
    torch.cuda.synchronize()
    codes, scale = quantised(W)
    ref = torch.full((M, N), 7.0, dtype=torch.bfloat16)
    for e in range(E):
        m, n = slice(off[e], off[e + 1]), slice(e * N, (e + 1) * N)
        ref[m] = product(X[m], codes[n], scale[n])
    assert torch.equal(Y.cpu(), ref)


def test_empty_batch(q):
    w = q.quantize_int8(rows(16, 64, 1, torch.float32).cuda())
    assert q.linear_int8(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), w).shape == (0, 16)


def test_captured_replay_and_other_stream(q):
    X, W = rows(40, 512, 1).cuda(), rows(520, 512, 2, torch.float32, 0.02)
    w = q.quantize_int8(W.cuda())
    q.set_check_device_status(False)
    ws = torch.empty(q.workspace_bytes_int8(40, 520, 512), dtype=torch.uint8, device="cuda")
    q.linear_int8(X, w, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = q.linear_int8(X, w, ws=ws)
    X.copy_(rows(40, 512, 9))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y.cpu(), product(X.cpu(), *quantised(W)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        Y2 = q.linear_int8(X, w)
    s.synchronize()
    assert torch.equal(Y, Y2)


def test_train_merge_and_serve_a_layer_of_experts(q):
    """The operators as they are used: a router's ids to an order, the experts'
    forward in NF4 with adapters, the adapters merged into 16 bits, the merged
    experts in 8 bits, their product on the same rows. What 8 bits lose is at
    most half a step per factor: |Y8 - Y| <= sum over k of (|x| dw + |w| dx + dx dw)
    with dx = max|x| / 254, dw = max|w| / 254, plus the bf16 roundings of the
    merged weight, of Y and of Y8 (2^-8 each)."""
    E, N, K, r, T = 4, 256, 256, 16, 75          # N K / 64 is a multiple of 256: the stack splits into experts
    cfg = synth.custom(N=E * N, K=K, M=2 * T, r=r, seed_base=900)
    g = torch.Generator().manual_seed(4)
    tokens = torch.randn(T, K, generator=g).bfloat16().cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:2] for _ in range(T)]).to(torch.int32).reshape(-1).cuda()
    A = torch.randn(E * r, K, generator=g).mul_(K ** -0.5).bfloat16().cuda()
    B = torch.randn(E * N, r, generator=g).mul_(0.05).bfloat16().cuda()
    w = q.quantize_nf4(synth.weight(cfg).cuda())
    order, offsets = q.expert_order(ids, E)
    X = tokens[(order // 2).long()]
    Y, sT = q.linear_fwd_experts(X, w, A, B, offsets, E, cfg.alpha)
    dX, dA, dB = q.linear_bwd_experts(torch.ones_like(Y), X, w, A, B, offsets, E, cfg.alpha, sT=sT)
    assert torch.isfinite(dA).all() and torch.isfinite(dB).all() and torch.isfinite(dX.float()).all()
    merged = torch.cat([q.merge_lora(q.expert_weight(w, e, E), A[e * r:(e + 1) * r], B[e * N:(e + 1) * N], cfg.alpha)
                        for e in range(E)])
    Y8 = q.linear_int8_experts(X, q.quantize_int8(merged), offsets, E)
    torch.cuda.synchronize()
    off = offsets.tolist()
    for e in range(E):
        m = slice(off[e], off[e + 1])
        x, wm = X[m].double(), merged[e * N:(e + 1) * N].double()
        dx, dw = x.abs().amax(1, keepdim=True) / 254, wm.abs().amax(1, keepdim=True).t() / 254
        y = Y[m].double()
        tol = x.abs().sum(1, keepdim=True) * dw + dx * wm.abs().sum(1)[None] + K * dx * dw
        tol += 2.0 ** -8 * (x.abs() @ wm.abs().t() + 3 * y.abs()) + 1e-2 * y.abs().max()
        assert torch.all((Y8[m].double() - y).abs() <= tol), e
    # and back to the router's order: every token's two rows
    back = torch.empty_like(Y8)
    back[order.long()] = Y8
    assert torch.equal(back.reshape(T, 2, N)[0, 0], Y8[(order == 0).nonzero()[0, 0]])


@pytest.mark.parametrize("tile,counts,N,K", [
    (64, [64, 64, 64], 264, 8208), (64, [20] * 75, 520, 1040), (64, [16, 17, 64, 65, 256, 257, 300, 1], 2056, 4112),
    (256, [90] * 6, 5000, 336), (256, [16, 17, 64, 65, 256, 257, 300, 1], 4104, 336), (256, [48, 15, 160, 129, 0, 256], 10248, 336),
    (512, [512, 513, 100, 257], 12808, 208), (512, [288, 289, 320, 31], 12808, 336)])
def test_tiles_bit_exact(q, tile, counts, N, K):
    """Every tile size, with counts around the granularities of its tokens, a weight
    tile that N ends in and a reduction that is no whole number of steps; rows of
    nobody on both sides."""
    E, M = len(counts), sum(counts) + 5
    assert q.tile_rows_int8(M, N, K, E) == tile
    X, W = rows(M, K, M), rows(E * N, K, N, torch.float32, 0.02)
    X[:2], X[M - 3:] = float("nan"), float("inf")
    off = np.concatenate([[0], np.cumsum(counts)]) + 2
    w = q.quantize_int8(W.cuda())
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    Y = [torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for y in Y:
        q.linear_int8_experts(X.cuda(), w, offsets, E, Y=y)
    codes, scale = quantised(W)
    ref = torch.full((M, N), 7.0, dtype=torch.bfloat16)
    for e in range(E):
        m, n = slice(off[e], off[e + 1]), slice(e * N, (e + 1) * N)
        ref[m] = product(X[m], codes[n], scale[n])
    for y in Y:
        assert torch.equal(y.cpu(), ref)


@pytest.mark.parametrize("tile,M,N,K", [(64, 100, 1000, 336), (256, 200, 40000, 144), (256, 130, 40008, 336),
                                        (512, 600, 5000, 336), (512, 257, 40008, 144)])
def test_dense_tiles_bit_exact(q, tile, M, N, K):
    assert q.tile_rows_int8(M, N, K) == tile
    X, W = rows(M, K, M + 1), rows(N, K, N + 2, torch.float32, 0.02)
    Y = q.linear_int8(X.cuda(), q.quantize_int8(W.cuda()))
    assert torch.equal(Y.cpu(), product(X, *quantised(W)))


def test_more_rows_than_an_int_counts_threads(q):
    """A CTA of 128 threads per row: 2^24 rows and some have more than 2^31
    threads."""
    M, N, K = (1 << 24) + 137, 8, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    W = torch.randn(N, K, generator=g, device="cuda") * 0.02
    w, rows8 = q.quantize_int8(W), q.quantize_int8(X)
    Y = q.linear_int8(X, w)
    for m in (slice(0, 1 << 20), slice((1 << 23) - 300, (1 << 23) + 300), slice((1 << 24) - 300, M)):
        x = X[m].cpu()
        codes, scale = quantised(x)
        assert torch.equal(rows8.codes[m].cpu(), codes) and torch.equal(rows8.scale[m].cpu(), scale)
        assert torch.equal(Y[m].cpu(), product(x, *quantised(W.cpu())))


@pytest.mark.parametrize("tile,counts,N,K", [(64, [9], 8, 4096), (64, [40], 520, 512), (256, [90] * 6, 5000, 336),
                                             (512, [1000], 12808, 256)], ids=["64_shared", "64", "256", "512"])
def test_scales_whose_product_is_no_normal_number(q, tile, counts, N, K):
    """Tiny and huge rows on both sides: xs ws leaves fp32's normal range where the
    sum times both does not, and a sum of zero stays zero. Where the product is
    normal the bits are those of the definition; elsewhere the sum's rounding and
    two products (2^-24 each) and the bf16 result (2^-8), or half of the least
    bf16 step, 2^-134, and overflow to infinity."""
    E, M = len(counts), sum(counts)
    assert q.tile_rows_int8(M, N, K, E) == tile
    X, W = rows(M, K, M + 3), rows(E * N, K, N + 4, torch.float32)
    X[0::7] *= 2.0 ** -76
    W[0::5] *= 2.0 ** -70
    X[1::7] *= 2.0 ** 76
    W[1::5] *= 2.0 ** 70
    X[1::7] = X[1, :1].abs()                     # equal tokens against alternating signs: sums of zero
    W[1::5] = W[1, :1].abs() * (1 - 2.0 * (torch.arange(K) % 2))
    w = q.quantize_int8(W.cuda())
    off = np.concatenate([[0], np.cumsum(counts)])
    Y = q.linear_int8(X.cuda(), w) if E == 1 else q.linear_int8_experts(
        X.cuda(), w, torch.tensor(off, dtype=torch.int32, device="cuda"), E)
    codes, scale = quantised(W)
    odd = 0
    for e in range(E):
        m, n = slice(off[e], off[e + 1]), slice(e * N, (e + 1) * N)
        qx, xs = quantised(X[m])
        s, p = qx.double() @ codes[n].double().t(), xs[:, None] * scale[n][None]
        normal = (p >= 2.0 ** -126) & torch.isfinite(p)
        got = Y[m].cpu()
        assert torch.equal(got[normal], product(X[m], codes[n], scale[n])[normal]), e
        ref = s * xs.double()[:, None] * scale[n].double()[None]
        big = ref.abs() >= 3.4e38                # above the largest bf16 number, 3.39e38
        assert torch.equal(got[~normal & big].double(), ref[~normal & big].sign() * float("inf")), e
        ok = (got.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -22) * ref.abs() + 2.0 ** -134
        assert ok[~normal & ~big].all(), (e, int((~ok & ~normal & ~big).sum()))
        odd += int((~normal).sum())
    assert odd > 0
