"""Workloads of the dropout and gated feed-forward operators.

Three operators of a finetuning step over frozen 4-bit weights, each with the
calls a training or serving program makes:

  dropout        Y = X * keep / (1 - p), the keep mask recomputed from a
                 counter (Philox-4x32-10), never stored; the gradient is the
                 same call on dY
  linear         the 4-bit linear (or fused projection) whose adapter reads
                 dropout(X): forward, and backward to dX, dA, dB
  gated          gate and up projections with their adapters, the activation
                 and the product, H = act(X Wg'^T + ...) * (X Wu'^T + ...):
                 forward (with or without the pre-activations kept for the
                 backward), and backward to dX, dA, dB

``own`` False computes a pass in its plain form, elementary torch operations
in fp32 rounded once at the end; ``own`` True makes the library's calls.
Tensors are synthetic and seeded; a quantized weight is drawn as N(0, 0.02)
and stored in the library's NF4 layout (64-element blocks, two codes a byte,
8-bit block constants in groups of 256).
"""
import math

import numpy as np
import torch

own = False

NF4 = (-1.0, -0.6961928009986877, -0.5250729322433472, -0.39491742849349976, -0.2844413220882416,
       -0.18477340042591095, -0.09104997664690018, 0.0, 0.07958031445741653, 0.16093014180660248,
       0.24611225724220276, 0.3379151225090027, 0.4407097399234772, 0.5626168847084045, 0.722956657409668, 1.0)
STEPS = 32768  # the drop probability is a whole number of 2^-15


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # the residual of a handful of sequences' last tokens: launch latency
        {"name": "dropout_64k_bf16", "op": "dropout", "n": 16 * 4096, "dtype": "bf16", "p": 0.1},
        # the residual stream of 16384 tokens of an 8192-wide model
        {"name": "dropout_128m_bf16", "op": "dropout", "n": 16384 * 8192, "dtype": "bf16", "p": 0.05},
        # an fp32 tensor whose length is no multiple of a vector
        {"name": "dropout_33m_odd_fp32", "op": "dropout", "n": 33554467, "dtype": "fp32", "p": 0.25},
        # the smallest training call: 16 tokens through a 256 x 256 linear
        {"name": "linear_fwd_tiny", "op": "linear_fwd", "M": 16, "nseg": 1, "S": 256, "K": 256, "r": 8, "p": 0.1},
        # LLaMA-7B attention output projection, 2048 tokens
        {"name": "linear_fwd_7b_o", "op": "linear_fwd", "M": 2048, "nseg": 1, "S": 4096, "K": 4096, "r": 64, "p": 0.05},
        # one 4096 x 4096 linear with a low-rank adapter, 2048 tokens
        {"name": "linear_bwd_4096_r16", "op": "linear_bwd", "M": 2048, "nseg": 1, "S": 4096, "K": 4096, "r": 16, "p": 0.1},
        # LLaMA-7B q/k/v as one weight, a batch whose tokens end inside a tile
        {"name": "linear_bwd_7b_qkv_ragged", "op": "linear_bwd", "M": 1531, "nseg": 3, "S": 4096, "K": 4096, "r": 64, "p": 0.05},
        # serving: one token through the LLaMA-7B feed-forward's gate and up
        {"name": "gated_fwd_7b_m1", "op": "gated_fwd", "M": 1, "F": 11008, "K": 4096, "r": 64, "p": 0.0, "keep": False},
        # serving: a batch of 48 sequences, LLaMA-65B
        {"name": "gated_fwd_65b_m48", "op": "gated_fwd", "M": 48, "F": 22016, "K": 8192, "r": 64, "p": 0.0, "keep": False},
        # training: 2048 tokens, LLaMA-65B, pre-activations kept, adapter dropout
        {"name": "gated_fwd_65b_train", "op": "gated_fwd", "M": 2048, "F": 22016, "K": 8192, "r": 64, "p": 0.05, "keep": True},
        # its backward on LLaMA-7B, ragged batch, no dropout
        {"name": "gated_bwd_7b_ragged", "op": "gated_bwd", "M": 1997, "F": 11008, "K": 4096, "r": 64, "p": 0.0},
        # the largest: the backward of the LLaMA-65B training call
        {"name": "gated_bwd_65b_train", "op": "gated_bwd", "M": 2048, "F": 22016, "K": 8192, "r": 64, "p": 0.05},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dropout", "linear_fwd", "linear_bwd", "gated_fwd", "gated_bwd"])
    p = round(rng.uniform(0.01, 0.5), 3)
    if op == "dropout":
        dtype = rng.choice(["bf16", "fp32"])
        return {"op": op, "n": _log(rng, 2000, (1 << 27) if dtype == "bf16" else (1 << 26)), "dtype": dtype, "p": p}
    r = rng.choice([8, 16, 24, 32, 40, 64])
    K = 64 * _log(rng, 2, 128)
    M = _log(rng, 1, 2048)
    if op.startswith("linear"):
        return {"op": op, "M": M, "nseg": rng.choice([1, 2, 3]), "S": 256 * _log(rng, 1, 32), "K": K, "r": r, "p": p}
    F = 256 * _log(rng, 1, 86)
    p = rng.choice([0.0, p])
    if op == "gated_fwd":
        return {"op": op, "M": M, "F": F, "K": K, "r": r, "p": p, "keep": rng.choice([False, True])}
    return {"op": op, "M": M, "F": F, "K": K, "r": r, "p": p}


def _dims(case):
    """M, N, K, nseg of a case's weight."""
    if case["op"].startswith("linear"):
        return case["M"], case["nseg"] * case["S"], case["K"], case["nseg"]
    return case["M"], 2 * case["F"], case["K"], 2


def work(case):
    op = case["op"]
    if op == "dropout":
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * e * case["n"], "flops": case["n"]}
    M, N, K, nseg = _dims(case)
    r, rt = case["r"], case["r"] * nseg
    weight = N * K * (0.5 + 1 / 64 + 4 / 16384)
    adapters = 2 * (rt * K + N * r)
    base = 2 * M * N * K
    up, down = 2 * M * rt * K, 2 * M * N * r  # X A^T (or G A, G^T X) and U B^T (or dY B, dY^T U)
    if op == "linear_fwd":
        return {"bytes": weight + adapters + 2 * M * (K + N), "flops": base + up + down}
    if op == "linear_bwd":
        return {"bytes": weight + adapters + 2 * M * (N + K) + 2 * M * K + adapters, "flops": base + 3 * up + 2 * down}
    F = N // 2
    if op == "gated_fwd":
        out = 2 * M * F + (2 * M * N if case["keep"] else 0)
        return {"bytes": weight + adapters + 2 * M * K + out, "flops": base + up + down + 6 * M * F}
    return {"bytes": weight + adapters + 2 * M * (F + N + K) + 2 * M * K + adapters,
            "flops": base + 3 * up + 2 * down + 12 * M * F}


# --------------------------------------------------------------------------- inputs
def _weight(N, K, gen, dev):
    """An N(0, 0.02) weight in the library's storage: codes, 8-bit block constants, their scales and offset."""
    nb = N * K // 64
    codes = torch.empty(N * K // 2, dtype=torch.uint8, device=dev)
    absmax = torch.empty(nb, dtype=torch.float32, device=dev)
    edges = torch.tensor([(a + b) / 2 for a, b in zip(NF4, NF4[1:])], dtype=torch.float32, device=dev)
    step = 1 << 20  # blocks at a time
    for b in range(0, nb, step):
        e = min(nb, b + step)
        w = torch.randn(e - b, 64, device=dev, generator=gen) * 0.02
        a = w.abs().amax(dim=1)
        c = torch.bucketize(w / a[:, None], edges).to(torch.uint8)
        codes[b * 32:e * 32] = ((c[:, 0::2] << 4) | c[:, 1::2]).reshape(-1)
        absmax[b:e] = a
    offset = absmax.double().mean().float().reshape(1)
    d = absmax - offset
    pad = torch.zeros(-nb % 256, device=dev)
    c1 = torch.cat([d, pad]).reshape(-1, 256).abs().amax(dim=1)
    q8 = (torch.round(d / c1.repeat_interleave(256)[:nb] * 127) + 127).to(torch.uint8)
    return {"rows": N, "cols": K, "codes": codes, "q8": q8, "c1": c1, "offset": offset}


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 17)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device=dev, generator=gen) * std).to(torch.bfloat16)

    st = {"case": dict(case), "seed": seed * 1000003 + 12345, "offset": 3 + seed % 1000}
    if case["op"] == "dropout":
        X = torch.randn(case["n"], device=dev, generator=gen)
        st["X"] = X if case["dtype"] == "fp32" else X.to(torch.bfloat16)
        return st
    M, N, K, nseg = _dims(case)
    r = case["r"]
    st["w"] = _weight(N, K, gen, dev)
    st["scale"] = 16.0 / r
    st["X"] = normal(M, K)
    st["A"] = normal(nseg * r, K, std=1.0 / r)
    st["B"] = normal(N, r, std=0.05)  # an adapter in mid-training
    if case["op"] == "linear_bwd":
        st["dY"] = normal(M, N)
    if case["op"] == "gated_bwd":
        st["dH"] = normal(M, N // 2)
        # the kept pre-activations of a forward: about N(0, 0.02 sqrt(K))
        st["GU"] = normal(M, N, std=0.02 * math.sqrt(K))
    if own:
        import bit_nf4_quantized_08_b200 as Q
        w = st["w"]
        st["nf4"] = Q.NF4Weight(N, K, True, w["codes"], absmax_q8=w["q8"], absmax_scale=w["c1"],
                                absmax_offset=w["offset"])
        bwd = case["op"].endswith("bwd")
        if case["op"].startswith("linear"):
            need = Q.qlora_fused_linear_dropout_workspace(M, st["nf4"], nseg, r, bwd)
        else:
            need = Q.qlora_gated_linear_workspace(M, st["nf4"], r, bwd)
        st["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    return st


# --------------------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    op = case["op"]
    if op == "dropout":
        X = st["X"]
        keep, up = _keep(X.numel(), case["p"], st["seed"], st["offset"], X.device)
        return torch.where(keep, X.float() * up, 0.0).to(X.dtype)
    M, N, K, nseg = _dims(case)
    W = _dequant(st["w"])
    X, A, B = st["X"].float(), st["A"].float(), st["B"].float()
    keep, up = _keep(M * K, case["p"], st["seed"], st["offset"], X.device)
    s = st["scale"] * up
    Xd = torch.where(keep.view(M, K), X, 0.0) if case["p"] else X
    if op.endswith("fwd"):
        U = (Xd @ A.t()) * s
        Y = X @ W.t() + _segments(U, B, nseg)
        if op == "linear_fwd":
            return Y.to(torch.bfloat16)
        g, u = Y[:, :N // 2], Y[:, N // 2:]
        H = (g * torch.sigmoid(g) * u).to(torch.bfloat16)
        return {"H": H, "GU": Y.to(torch.bfloat16)} if case["keep"] else H
    if op == "linear_bwd":
        dY = st["dY"].float()
    else:
        dH, GU = st["dH"].float(), st["GU"].float()
        g, u = GU[:, :N // 2], GU[:, N // 2:]
        sig = torch.sigmoid(g)
        dY = torch.cat([dH * u * (sig * (1.0 + g * (1.0 - sig))), dH * (g * sig)], dim=1)
    S, r = N // nseg, case["r"]
    G = torch.cat([dY[:, i * S:(i + 1) * S] @ B[i * S:(i + 1) * S] for i in range(nseg)], dim=1) * s
    U = (Xd @ A.t()) * s
    dL = G @ A
    if case["p"]:
        dL = torch.where(keep.view(M, K), dL, 0.0)
    dX = dY @ W + dL
    dA = G.t() @ Xd
    dB = torch.cat([dY[:, i * S:(i + 1) * S].t() @ U[:, i * r:(i + 1) * r] for i in range(nseg)], dim=0)
    return {"dX": dX.to(torch.bfloat16), "dA": dA.to(torch.bfloat16), "dB": dB.to(torch.bfloat16)}


def _segments(U, B, nseg):
    """Each row segment of B times its own columns of U, side by side."""
    S, r = B.shape[0] // nseg, B.shape[1]
    return torch.cat([U[:, i * r:(i + 1) * r] @ B[i * S:(i + 1) * S].t() for i in range(nseg)], dim=1)


def _keep(n, p, seed, offset, dev):
    """Keep mask of elements 0..n-1 and the factor of the kept ones.

    Philox-4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2,
    3", 2011) with the seed as key and (block number, offset) as counter: a
    block gives eight 15-bit numbers, the low then the high half of each of
    its four words, and element e is number e % 8 of block e // 8.  It is kept
    if the number is at least T = round(32768 p)."""
    T = int(math.floor(p * STEPS + 0.5))
    if T == 0:
        return torch.ones(n, dtype=torch.bool, device=dev), 1.0
    low = 0xFFFFFFFF
    block = torch.arange((n + 7) // 8, dtype=torch.int64, device=dev)
    c0, c1 = block & low, block >> 32
    c2, c3 = torch.full_like(block, offset & low), torch.full_like(block, (offset >> 32) & low)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64-bit products, modulo 2^64
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], dim=1)
    numbers = torch.stack([words & 0x7FFF, (words >> 16) & 0x7FFF], dim=2).reshape(-1)[:n]
    return numbers >= T, STEPS / (STEPS - T)


def _dequant(w):
    """The bf16 weight values the layer multiplies with, as fp32 [rows, cols]."""
    dev = w["codes"].device
    table = torch.tensor(NF4, dtype=torch.float32, device=dev)
    pairs = torch.stack([table.repeat_interleave(16), table.repeat(16)], dim=1)  # [byte] -> two values
    t8 = torch.arange(-127, 128, dtype=torch.float32, device=dev) / 127.0
    nb = w["q8"].numel()
    a = t8[w["q8"].long()] * w["c1"].repeat_interleave(256)[:nb] + w["offset"]
    v = pairs[w["codes"].int()].view(nb, 64) * a[:, None]
    return v.to(torch.bfloat16).float().view(w["rows"], w["cols"])


def _run_own(st, case):
    import bit_nf4_quantized_08_b200 as Q
    op = case["op"]
    drop = Q.Dropout(case["p"], st["seed"], st["offset"]) if case["p"] else None
    if op == "dropout":
        return Q.qlora_dropout(st["X"], drop)
    w, X, A, B, s, ws = st["nf4"], st["X"], st["A"], st["B"], st["scale"], st["ws"]
    if op == "linear_fwd":
        return Q.qlora_fused_linear_dropout_fwd(X, w, case["nseg"], A, B, s, drop, ws=ws)
    if op == "gated_fwd":
        H, GU = Q.qlora_gated_linear_fwd(X, w, A, B, s, act="silu", dropout=drop, want_gu=case["keep"], ws=ws)
        return {"H": H, "GU": GU} if case["keep"] else H
    if op == "linear_bwd":
        dX, dA, dB = Q.qlora_fused_linear_dropout_bwd(st["dY"], X, w, case["nseg"], A, B, s, drop, ws=ws,
                                                      grad_dtype=torch.bfloat16)
    else:
        dX, dA, dB = Q.qlora_gated_linear_bwd(st["dH"], X, st["GU"], w, A, B, s, act="silu", dropout=drop, ws=ws,
                                              grad_dtype=torch.bfloat16)
    return {"dX": dX, "dA": dA, "dB": dB}


# --------------------------------------------------------------------------- the definition in 64 bits
def _philox_keep(n, p, seed, offset):
    """Keep mask (numpy), 32-bit words in 64-bit unsigned arithmetic."""
    u = np.uint64
    T = int(math.floor(p * STEPS + 0.5))
    mask, sh = u(0xFFFFFFFF), u(32)
    c = np.arange((n + 7) // 8, dtype=np.uint64)
    x = [c & mask, c >> sh, np.full_like(c, offset & 0xFFFFFFFF), np.full_like(c, (offset >> 32) & 0xFFFFFFFF)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for i in range(10):
        k0, k1 = u((key[0] + i * 0x9E3779B9) & 0xFFFFFFFF), u((key[1] + i * 0xBB67AE85) & 0xFFFFFFFF)
        p0, p1 = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(p1 >> sh) ^ x[1] ^ k0, p1 & mask, (p0 >> sh) ^ x[3] ^ k1, p0 & mask]
    out = np.empty((c.size, 8), dtype=np.uint16)
    for j in range(4):
        out[:, 2 * j] = x[j] & u(0x7FFF)
        out[:, 2 * j + 1] = (x[j] >> u(16)) & u(0x7FFF)
    return out.reshape(-1)[:n] >= T


def _weight64(w, lo, hi):
    """Rows lo..hi-1 of the weight as the layer's bf16 values, in fp64."""
    K = w["cols"]
    dev = w["codes"].device
    b = w["codes"][lo * K // 2:hi * K // 2]
    nib = torch.stack([b >> 4, b & 15], dim=1).reshape(hi - lo, K).long()
    blk = torch.arange(lo * K // 64, hi * K // 64, device=dev)
    a = (w["q8"][blk].float() - 127) / 127.0
    a = a * w["c1"][blk // 256] + w["offset"]  # fp32, two roundings, as the format defines
    v = torch.take(torch.tensor(NF4, dtype=torch.float32, device=dev), nib) * a.repeat_interleave(64).view(hi - lo, K)
    return v.bfloat16().double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "dropout":
        n, T = case["n"], int(math.floor(case["p"] * STEPS + 0.5))
        keep = torch.from_numpy(_philox_keep(n, case["p"], st["seed"], st["offset"])).to(st["X"].device)
        return st["X"].double() * keep * (STEPS / (STEPS - T))
    if not torch.cuda.is_available():
        return None
    M, N, K, nseg = _dims(case)
    r, S, w = case["r"], N // nseg, st["w"]
    X, A, B = st["X"].double(), st["A"].double(), st["B"].double()
    s, mask = st["scale"], None
    if case["p"]:
        T = int(math.floor(case["p"] * STEPS + 0.5))
        mask = torch.from_numpy(_philox_keep(M * K, case["p"], st["seed"], st["offset"])).to(X.device).view(M, K)
        s = s * STEPS / (STEPS - T)
    Xd = X if mask is None else X * mask
    U = Xd.mm(A.t()) * s
    step = 4096
    if op.endswith("fwd"):
        Y = torch.empty(M, N, dtype=torch.float64, device=X.device)
        for lo in range(0, N, step):
            hi = min(N, lo + step)
            Y[:, lo:hi] = X.mm(_weight64(w, lo, hi).t())
        for i in range(nseg):
            Y[:, i * S:(i + 1) * S] += U[:, i * r:(i + 1) * r].mm(B[i * S:(i + 1) * S].t())
        if op == "linear_fwd":
            return Y
        g, u = Y[:, :S], Y[:, S:]
        H = g / (1.0 + torch.exp(-g)) * u
        return {"H": H, "GU": Y} if case["keep"] else H
    if op == "linear_bwd":
        dY = st["dY"].double()
    else:
        dH, g, u = st["dH"].double(), st["GU"][:, :S].double(), st["GU"][:, S:].double()
        e = torch.exp(-g)
        dY = torch.empty(M, N, dtype=torch.float64, device=X.device)
        dY[:, :S] = dH * u * (1.0 + e + g * e) / (1.0 + e) ** 2
        dY[:, S:] = dH * g / (1.0 + e)
    G = torch.empty(M, nseg * r, dtype=torch.float64, device=X.device)
    dB = torch.empty(N, r, dtype=torch.float64, device=X.device)
    for i in range(nseg):
        G[:, i * r:(i + 1) * r] = dY[:, i * S:(i + 1) * S].mm(B[i * S:(i + 1) * S]) * s
        dB[i * S:(i + 1) * S] = dY[:, i * S:(i + 1) * S].t().mm(U[:, i * r:(i + 1) * r])
    dX = G.mm(A)
    if mask is not None:
        dX = dX * mask
    for lo in range(0, N, step):
        hi = min(N, lo + step)
        dX += dY[:, lo:hi].mm(_weight64(w, lo, hi))
    return {"dX": dX, "dA": G.t().mm(Xd), "dB": dB}
