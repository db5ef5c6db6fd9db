"""Host checks of the expert and 8-bit calls, without a GPU: sizes, and bad
arguments rejected before any CUDA call."""
import ctypes

import pytest
import torch

P = 0x7000000  # fake, 16-byte aligned; never dereferenced on these paths


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_09_b200 import build
    build.build()
    import bit_nf4_quantized_09_b200 as q
    return q


def weight(q, N=4 * 512, K=512):
    return q.Nf4WeightC(P, P + 0x100000, P + 0x200000, P + 0x300000, N, K)


def test_workspaces(q):
    fwd = q.workspace_bytes_experts(q.OP_FWD, 100, 512, 512, 16, 4)
    bwd = q.workspace_bytes_experts(q.OP_BWD, 100, 512, 512, 16, 4)
    assert 0 < fwd < bwd
    for bad in ((q.OP_QUANTIZE, 100, 512, 512, 16, 4), (q.OP_FWD, -1, 512, 512, 16, 4), (q.OP_FWD, 1, 12, 512, 16, 4),
                (q.OP_FWD, 1, 512, 500, 16, 4), (q.OP_FWD, 1, 512, 512, 24, 4), (q.OP_FWD, 1, 512, 512, 16, 0),
                (q.OP_FWD, 1, 512, 512, 16, 513), (q.OP_FWD, 1 << 31, 512, 512, 16, 4)):
        assert q.workspace_bytes_experts(*bad) == 0, bad
    assert q.workspace_bytes_int8(100, 512, 528, 1) >= 100 * 528 + 400
    for bad in ((-1, 512, 512, 1), (1, 12, 512, 1), (1, 512, 520, 1), (1, 512, 131088, 1), (1, 512, 512, 0)):
        assert q.workspace_bytes_int8(*bad) == 0, bad


@pytest.mark.parametrize("N,K,r,E", [(512, 512, 16, 4), (11008, 4096, 64, 8), (8, 64, 8, 1), (264, 320, 8, 512),
                                     (2056, 1088, 32, 16)])
def test_workspaces_of_large_batches_serve_small_ones(q, N, K, r, E):
    L = q.lib()
    w = weight(q, N=E * N, K=K)
    w8 = q.Int8WeightC(P, P, E * N, K)
    sizes = [1, 2, 7, 8, 9, 15, 16, 17, 48, 63, 64, 65, 96, 97, 250, 700, 1500, 4000, 6145, 9000, 70000]
    last = [0, 0, 0]
    for M in sizes:
        now = [q.workspace_bytes_experts(q.OP_FWD, M, N, K, r, E), q.workspace_bytes_experts(q.OP_BWD, M, N, K, r, E),
               q.workspace_bytes_int8(M, N, K, E)]
        assert all(a >= b for a, b in zip(now, last)), (M, now, last)
        last = now
        # enough for the call itself, which ends on an injected failure
        q.set_option(q.OPT_FAIL_LAUNCHES, 3)
        got = [L.qlora_linear_fwd_experts(P, M, ctypes.byref(w), E, P, P, P, r, 16.0, P, None, P, now[0], None),
               L.qlora_linear_bwd_experts(P, P, M, ctypes.byref(w), E, P, P, P, r, 16.0, P, P, P, P, P, now[1], None),
               L.qlora_linear_int8_experts(P, M, ctypes.byref(w8), E, P, P, P, now[2], None)]
        q.set_option(q.OPT_FAIL_LAUNCHES, 0)
        assert got == [-6, -6, -6], (M, got)


def test_tile_rows(q):
    """Plans on both sides of the rules' borders, as measured in their comments, and 0
    for what the calls refuse."""
    f = lambda M, op=q.OP_FWD: q.tile_rows_experts(op, M, 4096, 4096, 8)  # noqa: E731
    assert [f(48), f(49), f(96), f(97), f(320)] == [8, 16, 16, 64, 64]
    assert f(600) in (64, 256) and f(1024) == 256 and f(4096) == 512
    assert f(48, q.OP_BWD) == 64
    assert q.tile_rows_int8(600, 4096, 4096, 8) == 256 and q.tile_rows_int8(64, 4096, 4096, 8) == 64
    assert q.tile_rows_int8(200, 11008, 4096) == 512 and q.tile_rows_int8(1, 22016, 8192) == 64
    for bad in ((q.OP_QUANTIZE, 9, 512, 512, 4), (q.OP_FWD, 0, 512, 512, 4), (q.OP_FWD, 9, 12, 512, 4), (q.OP_BWD, 9, 512, 500, 4),
                (q.OP_FWD, 9, 512, 512, 0), (q.OP_FWD, 1 << 31, 512, 512, 4)):
        assert q.tile_rows_experts(*bad) == 0, bad
    for bad in ((0, 512, 512, 1), (9, 12, 512, 1), (9, 512, 520, 1), (9, 512, 512, 513)):
        assert q.tile_rows_int8(*bad) == 0, bad


def test_forward_and_backward_refusals(q):
    L = q.lib()
    ws = q.workspace_bytes_experts(q.OP_FWD, 64, 512, 512, 16, 4)
    wsb = q.workspace_bytes_experts(q.OP_BWD, 64, 512, 512, 16, 4)

    def fwd(X=P, M=64, w=None, E=4, off=P, A=P, B=P, r=16, alpha=16.0, Y=P, sT=None, ws_=P, n=0):
        w = weight(q) if w is None else w
        return L.qlora_linear_fwd_experts(X, M, ctypes.byref(w), E, off, A, B, r, alpha, Y, sT, ws_, n, None)

    def bwd(dY=P, X=P, M=64, w=None, E=4, off=P, A=P, r=16, alpha=16.0, sT=None, dX=P, dA=P, dB=P, n=0):
        w = weight(q) if w is None else w
        return L.qlora_linear_bwd_experts(dY, X, M, ctypes.byref(w), E, off, A, P, r, alpha, sT, dX, dA, dB, P, n, None)

    for f in (fwd, bwd):
        assert f(E=0) == -1 and f(E=513) == -1
        assert f(E=3) == -2                              # 2048 rows over 3 experts
        assert f(w=weight(q, N=4 * 12)) == -2            # 12 rows per expert
        assert f(w=weight(q, K=500)) == -2
        assert f(off=None) == -1 and f(off=P + 2) == -3
        assert f(M=-1) == -2 and f(M=1 << 31) == -2
        assert f(r=24) == -4
        assert f(alpha=float("inf")) == -1
        assert f(X=None) == -1 and f(X=P + 2) == -3
        assert f(A=None) == -1
        assert f(sT=P + 8) == -3
    assert fwd(n=ws - 1) == -5 and bwd(n=wsb - 1) == -5
    assert fwd(Y=None) == -1 and fwd(ws_=None) == -1 and fwd(ws_=P + 8) == -3
    assert fwd(M=0, off=None) == 0                       # nothing to do
    assert bwd(dY=None) == -1 and bwd(dX=None) == -1 and bwd(dA=None) == -1 and bwd(dB=P + 4) == -3


def test_int8_refusals(q):
    L = q.lib()
    for entry in (L.qlora_quantize_int8, L.qlora_quantize_int8_bf16):
        assert entry(None, 8, 64, P, P, None) == -1
        assert entry(P, 0, 64, P, P, None) == -2
        assert entry(P, 8, 72, P, P, None) == -2         # K % 16
        assert entry(P, 8, 64, P + 8, P, None) == -3
    ws = q.workspace_bytes_int8(64, 512, 512, 4)

    def w8(N=2048, K=512, codes=P, scale=P):
        return q.Int8WeightC(codes, scale, N, K)

    def dense(X=P, M=64, w=None, Y=P, n=0):
        return L.qlora_linear_int8(X, M, ctypes.byref(w or w8()), Y, P, n, None)

    def experts(X=P, M=64, w=None, E=4, off=P, Y=P, n=0):
        return L.qlora_linear_int8_experts(X, M, ctypes.byref(w or w8()), E, off, Y, P, n, None)

    for f in (dense, experts):
        assert f(w=w8(codes=None)) == -1 and f(w=w8(scale=None)) == -1
        assert f(w=w8(codes=P + 8)) == -3
        assert f(w=w8(K=520)) == -2 and f(w=w8(N=12)) == -2 and f(w=w8(K=131088)) == -2
        assert f(M=-1) == -2 and f(M=1 << 31) == -2
        assert f(X=None) == -1 and f(X=P + 4) == -3 and f(Y=None) == -1
        assert f(n=ws - 1) == -5
        assert f(M=0) == 0
    assert experts(E=0) == -1 and experts(E=3) == -2 and experts(off=None) == -1 and experts(off=P + 1) == -3


def test_order_refusals(q):
    f = q.lib().qlora_expert_order
    assert f(P, 8, 0, P, P, None) == -1 and f(P, 8, 513, P, P, None) == -1
    assert f(P, -1, 4, P, P, None) == -2
    assert f(None, 8, 4, P, P, None) == -1 and f(P, 8, 4, None, P, None) == -1 and f(P, 8, 4, P, None, None) == -1
    assert f(P + 2, 8, 4, P, P, None) == -3


def test_injected_failures_reach_no_gpu(q):
    L = q.lib()
    w, w8 = weight(q), q.Int8WeightC(P, P, 2048, 512)
    calls = (lambda: L.qlora_linear_fwd_experts(P, 64, ctypes.byref(w), 4, P, P, P, 16, 16.0, P, None, P, 1 << 30, None),
             lambda: L.qlora_linear_bwd_experts(P, P, 64, ctypes.byref(w), 4, P, P, P, 16, 16.0, None, P, P, P, P, 1 << 30,
                                                None),
             lambda: L.qlora_linear_int8(P, 64, ctypes.byref(w8), P, P, 1 << 30, None),
             lambda: L.qlora_quantize_int8(P, 64, 64, P, P, None),
             lambda: L.qlora_expert_order(P, 64, 4, P, P, None))
    for call in calls:
        q.set_option(q.OPT_FAIL_LAUNCHES, 1)
        try:
            assert call() == -6
            assert q.get_option(q.OPT_FAIL_LAUNCHES) == 0
        finally:
            q.set_option(q.OPT_FAIL_LAUNCHES, 0)


def test_binding_refuses_wrong_tensors(q):
    """Shapes, types, strides and devices are checked before the library is
    called; tensors on the CPU are refused."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    E, N, K, r, M = 2, 64, 64, 8, 5
    w = q.NF4Weight(torch.zeros(E * N * K // 2, dtype=torch.uint8), torch.zeros(E * N, dtype=torch.uint8),
                    torch.zeros(1), torch.zeros(1), E * N, K)
    ok = dict(X=bf(M, K), w=w, A=bf(E * r, K), B=bf(E * N, r), offsets=i32(E + 1), E=E, alpha=16.0)
    bad = [dict(X=bf(M, K + 64)), dict(X=bf(M, K).float()), dict(X=bf(K, M).t()), dict(A=bf(E * r, K + 64)),
           dict(B=bf(E * N, 2 * r)), dict(offsets=i32(E)), dict(offsets=i32(E + 1).long()), dict(E=3), dict(E=0),
           dict(Y=bf(M, N + 8)), dict(sT=bf(M, r)), dict(ws=torch.zeros(1 << 20))]
    for change in bad + [{}]:                            # the last: everything fits but is not on a GPU
        with pytest.raises(q.QLoraError):
            q.linear_fwd_experts(**{**ok, **change})
    with pytest.raises(q.QLoraError):
        q.linear_bwd_experts(bf(M, N + 8), **ok)
    with pytest.raises(q.QLoraError):
        q.linear_bwd_experts(bf(M, N), sT=bf(M, r), **ok)
    with pytest.raises(q.QLoraError):
        q.expert_order(torch.zeros(4, dtype=torch.int64), 2)
    with pytest.raises(q.QLoraError):
        q.expert_order(i32(4), 2)
    w8 = q.Int8Weight(torch.zeros(N, K, dtype=torch.int8), torch.zeros(N), N, K)
    for X in (bf(M, K + 16), bf(M, K).float(), bf(M, K)):
        with pytest.raises(q.QLoraError):
            q.linear_int8(X, w8)
    with pytest.raises(q.QLoraError):
        q.linear_int8_experts(bf(M, K), w8, i32(3), 3)
    with pytest.raises(q.QLoraError):
        q.quantize_int8(torch.zeros(8, 64, dtype=torch.float16))
    with pytest.raises(q.QLoraError):
        q.quantize_int8(torch.zeros(8, 64))


def test_expert_weight_views(q):
    """One expert of a stack is a view where its constants start on a group of
    256 blocks; elsewhere it is refused."""
    def stack(N, K, dq):
        nb = 2 * N * K // 64
        codes = torch.arange(2 * N * K // 2, dtype=torch.int64).to(torch.uint8)
        if dq:
            return q.NF4Weight(codes, torch.zeros(nb, dtype=torch.uint8), torch.arange(-(-nb // 256)).float(),
                               torch.zeros(1), 2 * N, K)
        return q.NF4Weight(codes, None, None, None, 2 * N, K, absmax=torch.arange(nb).float())
    w = stack(256, 64, True)
    v = q.expert_weight(w, 1, 2)
    assert (v.N, v.K) == (256, 64) and v.s2.tolist() == [1.0] and v.codes.data_ptr() == w.codes.data_ptr() + 256 * 32
    v = q.expert_weight(stack(8, 64, False), 1, 2)
    assert v.absmax.tolist() == [float(i) for i in range(8, 16)]
    for bad in ((stack(128, 64, True), 1, 2), (w, 2, 2), (w, -1, 2), (w, 0, 3)):
        with pytest.raises(q.QLoraError):
            q.expert_weight(*bad)


@pytest.mark.parametrize("N,K", [((1 << 30) + 8, 64), (1 << 31, 64), ((1 << 32) - 8, 64), (8, (1 << 30) + 64),
                                 (8, 1 << 31), (64, 1 << 32)])
def test_more_columns_than_32_bit_numbers_hold(q, N, K):
    """Rows and columns of an expert are 32-bit numbers in the kernels, with room for
    a tile behind the last: wider weights are refused before anything runs."""
    L = q.lib()
    w = weight(q, N=N, K=K)
    for op in (q.OP_FWD, q.OP_BWD):
        assert q.workspace_bytes_experts(op, 4, N, K, 16, 1) == 0
    big = 1 << 62
    q.set_option(q.OPT_FAIL_LAUNCHES, 3)                 # nothing reaches a GPU where it is accepted
    try:
        assert L.qlora_linear_fwd_experts(P, 4, ctypes.byref(w), 1, P, P, P, 16, 16.0, P, None, P, big, None) == -2
        assert L.qlora_linear_bwd_experts(P, P, 4, ctypes.byref(w), 1, P, P, P, 16, 16.0, P, P, P, P, P, big, None) == -2
        if K <= 131072:
            w8 = q.Int8WeightC(P, P, N, K)
            assert L.qlora_linear_int8(P, 4, ctypes.byref(w8), P, P, big, None) == -2
            assert L.qlora_linear_int8_experts(P, 4, ctypes.byref(w8), 1, P, P, P, big, None) == -2
            assert q.workspace_bytes_int8(4, N, K) == 0
    finally:
        q.set_option(q.OPT_FAIL_LAUNCHES, 0)


def test_widest_weights_are_accepted(q):
    for N, K in ((1 << 30, 64), (8, 1 << 30)):
        assert q.workspace_bytes_experts(q.OP_FWD, 4, N, K, 16, 1) > 0
        assert q.workspace_bytes_experts(q.OP_BWD, 4, N, K, 16, 1) > 0
    assert q.workspace_bytes_int8(4, 1 << 30, 64) > 0


def test_quantiser_refuses_rows_it_cannot_number(q):
    """The quantiser numbers a row's vectors of eight in 32 bits: 2^33 columns."""
    L = q.lib()
    for entry in (L.qlora_quantize_int8, L.qlora_quantize_int8_bf16):
        for K, want in ((1 << 33, -6), ((1 << 33) + 16, -2), (1 << 34, -2), (1 << 40, -2)):
            q.set_option(q.OPT_FAIL_LAUNCHES, 1)
            try:
                assert entry(P, 1, K, P, P, None) == want, K
            finally:
                q.set_option(q.OPT_FAIL_LAUNCHES, 0)


def test_int8_weight_checks_replaced_tensors(q):
    """A weight keeps its C view while its tensors stay where they are; a tensor
    put in one's place at the same address, but strided, is refused as it is at
    the first call."""
    w8 = q.Int8Weight(torch.zeros(64, 64, dtype=torch.int8), torch.zeros(64), 64, 64)
    first = w8.c_view()
    assert w8.c_view() is first
    w8.codes = w8.codes.t()
    with pytest.raises(q.QLoraError):
        w8.c_view()
    w8.codes = w8.codes.t()
    w8.scale = torch.as_strided(w8.scale, (64,), (0,))
    with pytest.raises(q.QLoraError):
        w8.c_view()


@pytest.mark.parametrize("part,value,what", [
    ("codes", torch.zeros(64 * 64 - 1, dtype=torch.uint8), "codes"), ("qabsmax", torch.zeros(127, dtype=torch.uint8), "qabsmax"),
    ("s2", torch.zeros(0), "s2"), ("mean", torch.zeros(1, dtype=torch.float64), "mean"),
    ("s2", torch.zeros(1, device="meta"), "s2"), ("absmax", torch.zeros(127), "absmax")])
def test_parts_of_a_stacked_weight_are_checked(q, part, value, what):
    """A part that is too small, of another type or on another device would be read
    out of range by the kernels."""
    E, N, K, r, M = 2, 64, 64, 8, 5
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    parts = dict(codes=torch.zeros(E * N * K // 2, dtype=torch.uint8), qabsmax=torch.zeros(E * N, dtype=torch.uint8),
                 s2=torch.zeros(1), mean=torch.zeros(1), absmax=None)
    if part == "absmax":
        parts |= dict(qabsmax=None, s2=None, mean=None)
    w = q.NF4Weight(N=E * N, K=K, **{**parts, part: value})
    with pytest.raises(q.QLoraError, match=f"weight's {what}"):
        q.linear_fwd_experts(bf(M, K), w, bf(E * r, K), bf(E * N, r), torch.zeros(E + 1, dtype=torch.int32), E, 16.0)
    with pytest.raises(q.QLoraError, match=f"weight's {what}"):
        q.linear_bwd_experts(bf(M, N), bf(M, K), w, bf(E * r, K), bf(E * N, r), torch.zeros(E + 1, dtype=torch.int32), E, 16.0)
