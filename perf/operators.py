"""Measured cases of the expert and 8-bit operators.

Five operators: the row order of a batch by expert id; the forward and the
backward of a layer of experts with frozen NF4 weights and an adapter each
(rows grouped by expert, ragged); the product in 8-bit integers with a scale
for each token and output channel; and that product grouped by expert.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once), or, where ``own`` is set, through this repository's
package.
"""
from __future__ import annotations

import math
import statistics

import torch

own = False

BLOCK, GROUP = 64, 256


# ------------------------------------------------------------------ cases ---
def _experts(name, op, M, E, active, N, K, r, pad=0, dq=True, save=False):
    """M rows of which the last `pad` belong to no expert; `active` of the E
    experts have rows; N x K weights per expert, adapters of rank r; dq:
    stored with double quantisation."""
    return {"name": name, "op": op, "M": M, "E": E, "active": active, "N": N, "K": K, "r": r, "pad": pad, "dq": dq,
            "save": save}


def listed():
    return [
        # a router's ids in a decoding step: 8 requests, two experts each
        {"name": "order_decode", "op": "order", "M": 16, "E": 8},
        # the ids of a training batch over many small experts
        {"name": "order_batch", "op": "order", "M": 32768, "E": 64},
        # one request decoding a token: two experts of a gate projection
        _experts("fwd_token", "fwd", 2, 8, 2, 11008, 4096, 16),
        # 32 requests decoding, two experts each: a down projection
        _experts("fwd_decode", "fwd", 64, 8, 8, 4096, 11008, 16),
        # a short ragged prompt over narrow experts, padded at the end, fp32 constants
        _experts("fwd_ragged", "fwd", 1543, 16, 13, 2056, 4096, 8, pad=55, dq=False),
        # the forward of a training step, rank-r input kept for the backward
        _experts("fwd_train", "fwd", 8192, 8, 8, 11008, 4096, 64, save=True),
        # a short ragged backward
        _experts("bwd_ragged", "bwd", 777, 8, 7, 2056, 1088, 16, pad=9),
        # the backward of a training step over a down projection
        _experts("bwd_train", "bwd", 8192, 8, 8, 4096, 11008, 64),
        # one request decoding a token through a merged projection in 8 bits
        {"name": "int8_token", "op": "int8", "M": 1, "N": 22016, "K": 8192},
        # a long prompt through a merged projection
        {"name": "int8_prompt", "op": "int8", "M": 4096, "N": 11008, "K": 4096},
        # 32 requests decoding over merged experts
        _experts("int8_experts_decode", "int8_experts", 64, 8, 8, 4096, 4096, 0),
        # a long ragged prompt over merged experts
        _experts("int8_experts_prompt", "int8_experts", 8192, 16, 15, 4096, 4096, 0, pad=101),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["order", "fwd", "fwd", "bwd", "bwd", "int8", "int8_experts"])
    if op == "order":
        return {"op": op, "M": _log(rng, 1, 32768), "E": _log(rng, 1, 256)}
    if op == "int8":
        M = _log(rng, 1, 4096)
        return {"op": op, "M": M, "N": _log(rng, 8, 11008, 8), "K": _log(rng, 64, 4096, 16)}
    M, E = _log(rng, 1, 8192), _log(rng, 1, 16)
    pad = 0 if rng.random() < 0.5 else rng.randint(0, M // 8)
    active = rng.randint(1, max(1, min(E, M - pad)))
    N, K = _log(rng, 64, 4096, 8), _log(rng, 64, 4096, 64)
    case = _experts("", op, M, E, active, N, K, 0 if op == "int8_experts" else rng.choice([8, 16, 32, 64]), pad,
                    op == "int8_experts" or rng.random() < 0.7, op == "fwd" and rng.random() < 0.5)
    del case["name"]
    return case


# ------------------------------------------------------------- the inputs ---
def _levels():
    """The 16 NF4 levels: normal quantiles, an exact zero, ends -1 and 1."""
    q = statistics.NormalDist().inv_cdf
    top = 0.9677083
    v = [q(top - k * (top - 0.5) / 8) for k in range(8)] + [-q(top - k * (top - 0.5) / 7) for k in range(7)] + [0.0]
    return torch.tensor(sorted(v), dtype=torch.float64).div(max(v)).float().cuda()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _nf4(rows, K, dq, g):
    """An NF4 weight of normal values: packed codes (first of two in the high
    nibble) and its constants."""
    lv = _levels()
    mid = (lv[1:].double() + lv[:-1].double()).div(2).float()
    nb = rows * K // BLOCK
    w = torch.randn(nb, BLOCK, generator=g, device="cuda") * 0.02
    absmax = w.abs().amax(1)
    c = torch.bucketize(w / absmax[:, None], mid, out_int32=True).to(torch.uint8)
    codes = (c[:, ::2] << 4) | c[:, 1::2]
    if not dq:
        return {"codes": codes.reshape(-1), "absmax": absmax, "rows": rows, "K": K}
    mean = absmax.double().mean().float().reshape(1)
    ng = -(-nb // GROUP)
    d = torch.zeros(ng * GROUP, dtype=torch.float32, device="cuda")
    d[:nb] = absmax - mean
    s2 = d.reshape(ng, GROUP).abs().amax(1) / 448
    q = (d.reshape(ng, GROUP) / s2.clamp_min(1e-30)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return {"codes": codes.reshape(-1), "qabsmax": q.reshape(-1)[:nb].contiguous(), "s2": s2, "mean": mean,
            "rows": rows, "K": K}


def _counts(case, seed):
    """Rows of each expert: uneven, `active` of them not empty."""
    g = torch.Generator()
    g.manual_seed(int(seed))
    E, act, rows = case["E"], case["active"], case["M"] - case["pad"]
    share = torch.softmax(torch.randn(act, generator=g) * 0.4, 0)
    extra = torch.bincount(torch.multinomial(share, max(rows - act, 1), replacement=True, generator=g), minlength=act)
    n = torch.zeros(E, dtype=torch.int64)
    n[torch.randperm(E, generator=g)[:act]] = (extra if rows > act else torch.zeros_like(extra)) + 1
    return n


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    if op == "order":
        # uneven popularity; one id in a hundred names no expert (a dropped row)
        share = torch.softmax(randn(case["E"]), 0)
        ids = torch.multinomial(share, case["M"], replacement=True, generator=g).to(torch.int32)
        none = torch.rand(case["M"], generator=g, device="cuda") < 0.01
        s = {"op": op, "E": case["E"], "ids": torch.where(none, torch.full_like(ids, -1), ids)}
        return s
    M, N, K = case["M"], case["N"], case["K"]
    E = case.get("E", 1)
    s = {"op": op, "E": E, "N": N, "K": K, "X": randn(M, K).bfloat16()}
    if op != "int8":
        n = _counts(case, seed)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).to(torch.int32).cuda()
        s["cap"] = int(n.max())
    if op in ("int8", "int8_experts"):
        # outliers in a few channels, as activations have them
        s["X"][:, :: max(1, K // 8)] *= 8
        w = randn(E * N, K).mul_(0.02)
        a = w.abs().amax(1)
        s["wq"] = torch.round(w.mul_((127 / a)[:, None])).to(torch.int8)
        s["ws"] = a / 127
        s["Y"] = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        if own:
            import bit_nf4_quantized_09_b200 as q
            s["weight"] = q.Int8Weight(s["wq"], s["ws"], E * N, K)
            s["work"] = torch.empty(q.workspace_bytes_int8(M, N, K, E), dtype=torch.uint8, device="cuda")
        return s
    r = case["r"]
    s |= {"r": r, "alpha": 16.0, "save": case["save"], "w": _nf4(E * N, K, case["dq"], g),
          "A": randn(E * r, K).mul_(math.sqrt(2 / r) / math.sqrt(K)).bfloat16(), "B": randn(E * N, r).mul_(0.1).bfloat16()}
    if op == "fwd":
        s["Y"] = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        s["sT"] = torch.zeros(M, 2 * r, dtype=torch.bfloat16, device="cuda") if case["save"] else None
    else:
        s["dY"] = randn(M, N).bfloat16()
        s["dX"] = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
        # what the forward kept: s X A^T as the sum of two bf16 numbers
        rows, valid = _rows(s)
        t = torch.bmm(s["X"][rows].float(), s["A"].reshape(E, r, K).float().transpose(1, 2)) * (16.0 / r)
        hi = t.bfloat16()
        s["sT"] = torch.zeros(M, 2 * r, dtype=torch.bfloat16, device="cuda")
        s["sT"][rows[valid]] = torch.cat([hi, (t - hi.float()).bfloat16()], 2)[valid]
    if own:
        import bit_nf4_quantized_09_b200 as q
        w = s["w"]
        s["weight"] = q.NF4Weight(w["codes"], w.get("qabsmax"), w.get("s2"), w.get("mean"), E * N, K,
                                  absmax=w.get("absmax"))
        s["work"] = torch.empty(q.workspace_bytes_experts(q.OP_FWD if op == "fwd" else q.OP_BWD, M, N, K, r, E),
                                dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------- the plain forms ---
def _rows(s):
    """[E, cap] row numbers of each expert, padded, and which of them are its."""
    off = s["offsets"].long()
    rows = off[:-1, None] + torch.arange(s["cap"], device="cuda")
    valid = rows < off[1:, None]
    return torch.where(valid, rows, 0), valid


def _put(out, rows, valid, padded):
    """Writes the experts' rows of `padded` [E, cap, C] to their places in `out`."""
    at = torch.where(valid, rows, len(out))  # padding goes to a row behind the last
    big = torch.cat([out, out[:1]])
    big[at.reshape(-1)] = padded.reshape(-1, padded.shape[-1]).to(out.dtype)
    out.copy_(big[:-1])
    return out


def _dequantised(w):
    """The weight in fp32: level times constant, rounded to bf16 as the format says."""
    if "absmax" in w:
        c = w["absmax"]
    else:
        group = torch.arange(len(w["qabsmax"]), device="cuda") // GROUP
        e = w["qabsmax"].view(torch.float8_e4m3fn).double()
        c = (e * w["s2"].double()[group] + w["mean"].double()).float()
    code = torch.stack([w["codes"] >> 4, w["codes"] & 15], 1).reshape(-1, BLOCK).int()
    return (_levels()[code] * c[:, None]).bfloat16().float().reshape(w["rows"], w["K"])


def _plain_order(s):
    ids, E = s["ids"].long(), s["E"]
    key = torch.where((ids >= 0) & (ids < E), ids, E)
    hot = (key[:, None] == torch.arange(E + 1, device="cuda")).int()
    before = (torch.cumsum(hot, 0, dtype=torch.int32) - hot).gather(1, key[:, None])[:, 0]
    start = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), hot.sum(0).cumsum(0).int()])
    order = torch.empty(len(ids), dtype=torch.int32, device="cuda")
    order[(start[key] + before).long()] = torch.arange(len(ids), dtype=torch.int32, device="cuda")
    return order, start[:E + 1].contiguous()


def _plain_fwd(s):
    E, N, K, r = s["E"], s["N"], s["K"], s["r"]
    rows, valid = _rows(s)
    X = s["X"][rows].float()
    t = torch.bmm(X, s["A"].reshape(E, r, K).float().transpose(1, 2)) * (s["alpha"] / r)
    y = torch.bmm(X, _dequantised(s["w"]).reshape(E, N, K).transpose(1, 2))
    y += torch.bmm(t, s["B"].reshape(E, N, r).float().transpose(1, 2))
    Y = _put(s["Y"], rows, valid, y)
    if not s["save"]:
        return Y
    hi = t.bfloat16()
    return Y, _put(s["sT"], rows, valid, torch.cat([hi, (t - hi.float()).bfloat16()], 2))


def _plain_bwd(s):
    E, N, K, r = s["E"], s["N"], s["K"], s["r"]
    rows, valid = _rows(s)
    keep = valid[:, :, None]
    dY = torch.where(keep, s["dY"][rows].float(), 0)
    X = torch.where(keep, s["X"][rows].float(), 0)
    sT = torch.where(keep, s["sT"][rows].float(), 0)
    u = torch.bmm(dY, s["B"].reshape(E, N, r).float()) * (s["alpha"] / r)
    dx = torch.bmm(dY, _dequantised(s["w"]).reshape(E, N, K)) + torch.bmm(u, s["A"].reshape(E, r, K).float())
    dA = torch.bmm(u.transpose(1, 2), X).reshape(E * r, K)
    dB = torch.bmm(dY.transpose(1, 2), sT[:, :, :r] + sT[:, :, r:]).reshape(E * N, r)
    return _put(s["dX"], rows, valid, dx), dA, dB


def _quantised(x):
    """Codes round(127 x / max|x|), halves to even, and the scale max|x| / 127
    of each row; in 64 bits, where no quotient falls on the wrong side."""
    a = x.abs().amax(-1, keepdim=True).double()
    return torch.round(127 * x.double() / a.clamp_min(1e-300)).float(), (a / 127).float()


def _plain_int8(s):
    q, xs = _quantised(s["X"].float())
    if s["op"] == "int8":
        s["Y"].copy_(q @ s["wq"].float().t() * xs * s["ws"])
        return s["Y"]
    E, N, K = s["E"], s["N"], s["K"]
    rows, valid = _rows(s)
    y = torch.bmm(q[rows], s["wq"].reshape(E, N, K).float().transpose(1, 2))
    return _put(s["Y"], rows, valid, y * xs[rows] * s["ws"].reshape(E, 1, N))


def run(s):
    op = s["op"]
    if own:
        import bit_nf4_quantized_09_b200 as q
        if op == "order":
            return q.expert_order(s["ids"], s["E"])
        if op == "fwd":
            Y, sT = q.linear_fwd_experts(s["X"], s["weight"], s["A"], s["B"], s["offsets"], s["E"], s["alpha"],
                                         Y=s["Y"], sT=s["sT"], save_sT=s["save"], ws=s["work"])
            return (Y, sT) if s["save"] else Y
        if op == "bwd":
            return q.linear_bwd_experts(s["dY"], s["X"], s["weight"], s["A"], s["B"], s["offsets"], s["E"],
                                        s["alpha"], sT=s["sT"], dX=s["dX"], ws=s["work"])
        if op == "int8":
            return q.linear_int8(s["X"], s["weight"], Y=s["Y"], ws=s["work"])
        return q.linear_int8_experts(s["X"], s["weight"], s["offsets"], s["E"], Y=s["Y"], ws=s["work"])
    return {"order": _plain_order, "fwd": _plain_fwd, "bwd": _plain_bwd, "int8": _plain_int8,
            "int8_experts": _plain_int8}[op](s)


# ------------------------------------------------------------------- work ---
def work(case):
    op, M = case["op"], case["M"]
    if op == "order":
        return {"bytes": 8 * M + 4 * (case["E"] + 1), "flops": 0}
    N, K = case["N"], case["K"]
    rows, act = M - case.get("pad", 0), case.get("active", 1)
    if op in ("int8", "int8_experts"):
        return {"bytes": 2 * rows * (N + K) + act * N * (K + 4), "flops": 2 * rows * N * K}
    r, E = case["r"], case["E"]
    weight = act * N * K * (0.5 + (1 / BLOCK + 4 / (BLOCK * GROUP) if case["dq"] else 4 / BLOCK))
    if op == "fwd":
        kept = 4 * rows * r if case["save"] else 0
        return {"bytes": weight + 2 * rows * (N + K) + 2 * act * r * (N + K) + kept,
                "flops": 2 * rows * (N * K + r * (N + K))}
    # every expert's gradients are written, those of experts without rows as zeros
    return {"bytes": weight + 2 * rows * (N + 2 * K) + 4 * rows * r + 2 * act * r * (N + K) + 4 * E * r * (N + K),
            "flops": 2 * rows * (N * K + 3 * r * (N + K))}


# ------------------------------------------------- the definition in 64 bits ---
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "order":
        ids = [int(v) for v in s["ids"].cpu()]
        E = case["E"]
        key = [v if 0 <= v < E else E for v in ids]
        order = sorted(range(len(ids)), key=lambda m: key[m])
        return (torch.tensor(order, dtype=torch.int32),
                torch.tensor([sum(k < e for k in key) for e in range(E + 1)], dtype=torch.int32))
    M, N, K, E = case["M"], case["N"], case["K"], case.get("E", 1)
    off = s["offsets"].tolist() if op != "int8" else [0, M]
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
    if op in ("int8", "int8_experts"):
        Y = zeros(M, N)
        for e in range(E):
            x = s["X"][off[e]:off[e + 1]].double()
            top = x.abs().max(1, keepdim=True).values if len(x) else x[:, :1]
            q = (x * 127 / top).nan_to_num(0).round()
            rows = slice(e * N, (e + 1) * N)
            Y[off[e]:off[e + 1]] = (q @ s["wq"][rows].double().t()) * (top / 127) * s["ws"][rows].double()
        return Y
    r, w, scale = case["r"], s["w"], s["alpha"] / case["r"]
    lv, per = _levels().double(), N * K // BLOCK
    what = "Y" if op == "fwd" else "dX"
    out = zeros(M, N if op == "fwd" else K)
    kept, dA, dB = zeros(M, 2 * r), zeros(E * r, K), zeros(E * N, r)
    for e in range(E):
        if off[e] == off[e + 1]:
            continue
        at = torch.arange(e * per, (e + 1) * per, device="cuda")
        if case["dq"]:
            c = w["qabsmax"][at].view(torch.float8_e4m3fn).double() * w["s2"][at // GROUP].double() + w["mean"].double()
            c = c.float().double()
        else:
            c = w["absmax"][at].double()
        byte = w["codes"].reshape(-1, BLOCK // 2)[at].long()
        W = torch.empty(per, BLOCK, dtype=torch.float64, device="cuda")
        W[:, 0::2] = lv[byte // 16] * c[:, None]
        W[:, 1::2] = lv[byte % 16] * c[:, None]
        W = W.float().bfloat16().double().reshape(N, K)
        m = slice(off[e], off[e + 1])
        A, B, X = s["A"][e * r:(e + 1) * r].double(), s["B"][e * N:(e + 1) * N].double(), s["X"][m].double()
        if what == "Y":
            t = scale * (X @ A.t())
            out[m] = X @ W.t() + t @ B.t()
            kept[m, :r] = t.bfloat16().double()
            kept[m, r:] = t - kept[m, :r]
        else:
            dY = s["dY"][m].double()
            u = scale * (dY @ B)
            out[m] = dY @ W + u @ A
            dA[e * r:(e + 1) * r] = u.t() @ X
            dB[e * N:(e + 1) * N] = dY.t() @ (s["sT"][m, :r].double() + s["sT"][m, r:].double())
    if what == "dX":
        return out, dA, dB
    return (out, kept) if case["save"] else out
