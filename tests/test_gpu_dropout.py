"""GPU dropout: the elementwise call bit for bit against the published
generator, and the linear whose adapters read dropout(X) against fp64.

Tolerances of the linear: a bf16 rounding is off by at most 2^-8 of the value
and by 1.7e-3 of the norm over many values.  Y and dX carry their own rounding
and, in the adapter's term, that of U or G; dA and dB that of G or U and, in
bf16, their own: at most sqrt(2) * 1.7e-3 = 2.4e-3 of the norm, below the 5e-3
of the linear's tests; the largest error stays below 2 * 2^-8 = 7.9e-3 of the
largest value, below their 1e-2."""
import numpy as np
import pytest
import torch

from bit_nf4_quantized_08_b200 import workloads as wl
from conftest import assert_close_tol
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu


def _expected(O, x, p, seed, off):
    """fp32 product rounded to x's type where kept, +0 elsewhere (CPU tensors)."""
    keep = torch.from_numpy(O.dropout_keep(x.numel(), p, seed, off).reshape(x.shape))
    y = x.float() * np.float32(O.dropout_factor(p))
    return torch.where(keep, y, torch.zeros(())).to(x.dtype)


def _same_bits(a, b):
    it = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.contiguous().view(it), b.contiguous().view(it))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 2048, 2049, 100003, (1 << 21) + 5])
def test_dropout_bits(Q, O, cuda, dtype, n):
    x = torch.randn(n, generator=torch.Generator().manual_seed(n)).to(dtype)
    for p, seed, off in ((0.1, 5, 0), (0.5, (1 << 64) - 1, (1 << 64) - 1), (0.99, 1 << 40, 3)):
        y = Q.qlora_dropout(x.cuda(), Q.Dropout(p, seed, off)).cpu()
        assert _same_bits(y, _expected(O, x, p, seed, off)), (p, seed, off)


def test_dropout_grid_stride_and_sampled_blocks(Q, O, cuda):
    """More blocks than the grid holds in one pass, ragged end; sampled against the generator."""
    n = (1 << 26) + 13
    x = torch.ones(n, dtype=torch.bfloat16, device=cuda)
    y = Q.qlora_dropout(x, Q.Dropout(0.25, 77, 4))
    kept = (y != 0)
    assert abs(float(kept.float().mean()) - 0.75) < 6 * (0.75 * 0.25 / n) ** 0.5
    for first in (0, 8 * 1234567, (n // 8) * 8 - 800):
        m = min(800, n - first)
        assert np.array_equal(kept[first:first + m].cpu().numpy(), O.dropout_keep(m, 0.25, 77, 4, first))
    m = n - (n // 8) * 8
    assert np.array_equal(kept[-m:].cpu().numpy(), O.dropout_keep(m, 0.25, 77, 4, (n // 8) * 8))


def test_dropout_special_values_and_p0(Q, O, cuda):
    """Dropped NaN and infinities give +0; p = 0 (and any p that rounds to 0) is the identity."""
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0, 3e38, -1.5] * 50, dtype=dtype)
        keep = torch.from_numpy(O.dropout_keep(x.numel(), 0.5, 3, 9))
        y = Q.qlora_dropout(x.cuda(), Q.Dropout(0.5, 3, 9)).cpu()
        zero = torch.zeros(1, dtype=dtype)
        assert _same_bits(y[~keep], zero.expand(int((~keep).sum())))
        ref = (x.float() * 2).to(dtype)
        assert torch.equal(torch.isnan(y[keep]), torch.isnan(ref[keep]))
        fine = keep & ~torch.isnan(ref)
        assert torch.equal(y[fine], ref[fine])
        for p in (0.0, 2.0 ** -17):
            z = Q.qlora_dropout(x.cuda(), Q.Dropout(p, 3, 9)).cpu()
            assert torch.equal(torch.isnan(z), torch.isnan(x)) and torch.equal(z[~torch.isnan(x)], x[~torch.isnan(x)])


def test_dropout_in_place_guards_and_empty(Q, O, cuda):
    x = torch.randn(1003, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    g = Guarded((1003,), torch.bfloat16)
    g.t.copy_(x)
    Q.qlora_dropout(g.t, Q.Dropout(0.3, 8, 1), out=g.t)
    torch.cuda.synchronize()
    g.check("in place")
    assert _same_bits(g.t.cpu(), _expected(O, x, 0.3, 8, 1))
    e = torch.empty(0, device=cuda)
    assert Q.qlora_dropout(e, Q.Dropout(0.3, 8)).numel() == 0
    with pytest.raises(Q.QloraError) as err:
        Q.qlora_dropout(g.t[1:], Q.Dropout(0.3, 8))  # not 16-byte aligned
    assert err.value.status == Q.QLORA_ERR_INVALID_ARG


def test_dropout_gradient_is_the_same_call(Q, O, cuda):
    """<dropout(x), dy> == <x, dropout(dy)> in fp64: the call is its own transpose."""
    x, dy = torch.randn(2, 4096, device=cuda)
    d = Q.Dropout(0.2, 4, 4)
    a = (Q.qlora_dropout(x, d).double() * dy.double()).sum()
    b = (x.double() * Q.qlora_dropout(dy, d).double()).sum()
    # each product carries one fp32 rounding (2^-24) of its dropped-out factor
    bound = 2.0 ** -23 * float((x.double() * dy.double()).abs().sum()) * 1.25
    assert abs(float(a - b)) <= bound


def test_dropout_captured_graph_draws_new_masks(Q, O, cuda):
    x = torch.ones(4096, dtype=torch.bfloat16, device=cuda)
    ctr = torch.zeros(1, dtype=torch.int64, device=cuda)
    y = torch.empty_like(x)
    d = Q.Dropout(0.5, 21, 100, ctr)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        Q.qlora_dropout(x, d, out=y)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            Q.qlora_dropout(x, d, out=y)
            ctr += 1  # the program's own counter kernel, behind the call
    torch.cuda.current_stream().wait_stream(s)
    ctr.zero_()
    for i in range(4):
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal((y != 0).cpu().numpy(), O.dropout_keep(4096, 0.5, 21, 100 + i)), i


# --------------------------------------------------------------------------- the linear
def _setup(Q, M, nseg, S, K, r, seed, dq=True, zero_w=False, **fmt):
    N = nseg * S
    W = wl.weight(N, K, seed=seed, dtype=torch.bfloat16)
    if zero_w:
        W.zero_()
    # a large B: the adapter's terms are of the base's size
    inp = wl.fused_inputs(M, nseg, S, K, r, seed=seed, b_std=0.5)
    q = Q.qlora_nf4_quantize(W.cuda(), double_quant=dq, **fmt)
    Wd = wl.bits(Q.qlora_nf4_dequantize(q).cpu())  # bit-exact against the oracle in its own tests
    return q, inp, Wd


def _run(Q, q, inp, nseg, s, drop, grad_dtype=torch.float32, **kw):
    X, dY, A, B = (inp[k].cuda() for k in ("X", "dY", "A", "B"))
    Y = Q.qlora_fused_linear_dropout_fwd(X, q, nseg, A, B, s, drop)
    g = Q.qlora_fused_linear_dropout_bwd(dY, X, q, nseg, A, B, s, drop, grad_dtype=grad_dtype, **kw)
    torch.cuda.synchronize()
    assert Q.qlora_get_last_error() == 0
    return Y, g


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _check(Q, O, q, inp, Wd, nseg, s, drop, Y, g, tag):
    bits = [wl.bits(inp[k]) for k in ("X",)] + [Wd] + [wl.bits(inp[k]) for k in ("A", "B")]
    d = (drop.p, drop.seed, drop.offset)
    assert_close_tol(_f64(Y), O.dropout_linear_fwd(*bits, s, nseg, d), f"Y {tag}")
    ref = O.dropout_linear_bwd(inp["dY"].double().numpy(), *bits, s, nseg, d)
    for name, got, r in zip(("dX", "dA", "dB"), g, ref):
        if got is not None:
            assert_close_tol(_f64(got), r, f"{name} {tag}")


CASES = [
    # M, nseg, S, K, r: one token, ragged tiles, the small-token kernels, several column tiles
    (1, 1, 256, 64, 8), (3, 2, 256, 128, 8), (16, 1, 264, 192, 24), (17, 2, 512, 256, 16), (64, 3, 256, 320, 40),
    (65, 1, 136, 64, 8), (130, 2, 256, 448, 32), (300, 3, 256, 512, 64), (513, 1, 1000, 1088, 64),
    (1100, 2, 512, 576, 128), (200, 1, 512, 256, 256),
]


@pytest.mark.parametrize("M,nseg,S,K,r", CASES)
@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16], ids=["gfp32", "gbf16"])
def test_linear_dropout_parity(Q, O, cuda, M, nseg, S, K, r, grad_dtype):
    q, inp, Wd = _setup(Q, M, nseg, S, K, r, seed=70 + M)
    drop = Q.Dropout(0.3, 12345678901, 7)
    Y, g = _run(Q, q, inp, nseg, 2.0, drop, grad_dtype)
    assert g[1].dtype == grad_dtype and g[2].dtype == grad_dtype
    _check(Q, O, q, inp, Wd, nseg, 2.0, drop, Y, g, f"M={M} nseg={nseg} S={S} K={K} r={r}")


@pytest.mark.parametrize("M,K,r", [(7, 192, 16), (300, 320, 16), (600, 576, 64)])
def test_masked_adapter_gradient_exactly(Q, O, cuda, M, K, r):
    """With a zero weight dX is the adapter's term alone: exactly 0 where the mask drops, not 0 elsewhere."""
    q, inp, _ = _setup(Q, M, 1, 256, K, r, seed=5, zero_w=True)
    drop = Q.Dropout(0.4, 99, 1 << 33)
    _, (dX, _, _) = _run(Q, q, inp, 1, 2.0, drop)
    keep = O.dropout_keep(M * K, 0.4, 99, 1 << 33).reshape(M, K)
    assert np.array_equal((dX != 0).cpu().numpy(), keep)


@pytest.mark.parametrize("mode", [2, 3, 4, 6, 7, 8], ids=["streamk7", "single_cta_grid", "pair_streamk4", "serial_bwd",
                                                          "warp_mma", "tcgen05_small"])
@pytest.mark.parametrize("M", [12, 30, 600])
def test_linear_dropout_alternate_schedules(Q, O, cuda, mode, M):
    nseg, S, K, r = 3, 256, 512, 16
    q, inp, Wd = _setup(Q, M, nseg, S, K, r, seed=61)
    drop = Q.Dropout(0.1, 3, 3)
    Q.qlora_debug_inject(mode)
    try:
        Y, g = _run(Q, q, inp, nseg, 2.0, drop)
    finally:
        Q.qlora_debug_inject(0)
    _check(Q, O, q, inp, Wd, nseg, 2.0, drop, Y, g, f"mode {mode}")


def test_linear_dropout_without_dx_and_formats(Q, O, cuda):
    for fmt in (dict(dq=False), dict(blocksize=128, code_type="fp4", dq_type="e4m3")):
        q, inp, Wd = _setup(Q, 200, 2, 256, 256, 16, seed=62, **fmt)
        drop = Q.Dropout(0.2, 3, 4)
        Y, g = _run(Q, q, inp, 2, 2.0, drop, want_dx=False)
        assert g[0] is None
        _check(Q, O, q, inp, Wd, 2, 2.0, drop, Y, g, str(fmt))


def test_no_dropout_is_the_fused_linear(Q, cuda):
    """dropout None, p = 0 and p below 2^-16: the bits of qlora_fused_linear_fwd / _bwd."""
    for M in (9, 300):
        q, inp, _ = _setup(Q, M, 2, 256, 256, 16, seed=63)
        X, dY, A, B = (inp[k].cuda() for k in ("X", "dY", "A", "B"))
        ref = (Q.qlora_fused_linear_fwd(X, q, 2, A, B, 2.0), *Q.qlora_fused_linear_bwd(dY, X, q, 2, A, B, 2.0))
        for drop in (None, Q.Dropout(0.0, 1), Q.Dropout(2.0 ** -18, 1)):
            Y, g = _run(Q, q, inp, 2, 2.0, drop)
            assert all(_same_bits(a, b) for a, b in zip((Y, *g), ref))


def test_adapter_ignores_what_dropped_places_hold(Q, O, cuda):
    """NaN and infinities in dropped places of X reach neither dA nor dB."""
    for M in (40, 300):
        q, inp, _ = _setup(Q, M, 1, 256, 192, 16, seed=64)
        drop = Q.Dropout(0.5, 6, 6)
        keep = torch.from_numpy(O.dropout_keep(M * 192, 0.5, 6, 6).reshape(M, 192))
        _, (_, dA, dB) = _run(Q, q, inp, 1, 2.0, drop)
        X2 = inp["X"].clone()
        X2[~keep] = torch.tensor([float("nan"), float("inf")], dtype=torch.bfloat16).repeat(M * 192)[:int((~keep).sum())]
        _, (dX2, dA2, dB2) = _run(Q, q, dict(inp, X=X2), 1, 2.0, drop)
        assert _same_bits(dA, dA2) and _same_bits(dB, dB2) and bool(torch.isfinite(dX2).all())


def test_linear_dropout_empty_batch(Q, cuda):
    q, inp, _ = _setup(Q, 4, 2, 256, 128, 8, seed=65)
    A, B = inp["A"].cuda(), inp["B"].cuda()
    X, dY = torch.empty(0, 128, dtype=torch.bfloat16, device=cuda), torch.empty(0, 512, dtype=torch.bfloat16, device=cuda)
    assert Q.qlora_fused_linear_dropout_fwd(X, q, 2, A, B, 1.0, Q.Dropout(0.1, 1)).shape == (0, 512)
    for gd in (torch.float32, torch.bfloat16):
        dA, dB = torch.ones(16, 128, dtype=gd, device=cuda), torch.ones(512, 8, dtype=gd, device=cuda)
        Q.qlora_fused_linear_dropout_bwd(dY, X, q, 2, A, B, 1.0, Q.Dropout(0.1, 1), dA=dA, dB=dB, grad_dtype=gd)
        torch.cuda.synchronize()
        assert not dA.any() and not dB.any()


@pytest.mark.parametrize("M", [5, 40, 333])
def test_linear_dropout_guards_and_repeat(Q, cuda, M):
    """Outputs and workspace inside guard bytes; two runs give the same bits."""
    nseg, S, K, r = 2, 256, 320, 24
    q, inp, _ = _setup(Q, M, nseg, S, K, r, seed=66)
    X, dY, A, B = (inp[k].cuda() for k in ("X", "dY", "A", "B"))
    drop = Q.Dropout(0.15, 2, 2)
    outs = []
    for gd in (torch.float32, torch.bfloat16, torch.float32):
        G = {"Y": Guarded((M, nseg * S), torch.bfloat16), "dX": Guarded((M, K), torch.bfloat16),
             "dA": Guarded((nseg * r, K), gd), "dB": Guarded((nseg * S, r), gd),
             "wf": Guarded((Q.qlora_fused_linear_dropout_workspace(M, q, nseg, r, False),), torch.uint8),
             "wb": Guarded((Q.qlora_fused_linear_dropout_workspace(M, q, nseg, r, True),), torch.uint8)}
        Q.qlora_fused_linear_dropout_fwd(X, q, nseg, A, B, 2.0, drop, Y=G["Y"].t, ws=G["wf"].t)
        Q.qlora_fused_linear_dropout_bwd(dY, X, q, nseg, A, B, 2.0, drop, dX=G["dX"].t, dA=G["dA"].t, dB=G["dB"].t,
                                         ws=G["wb"].t, grad_dtype=gd)
        torch.cuda.synchronize()
        assert Q.qlora_get_last_error() == 0
        for k, g in G.items():
            g.check(k)
        outs.append([G[k].t.clone() for k in ("Y", "dX", "dA", "dB")])
    assert all(_same_bits(a, b) for a, b in zip(outs[0], outs[2]))
    # the bf16 gradients are the fp32 ones rounded once
    assert _same_bits(outs[0][2].to(torch.bfloat16), outs[1][2]) and _same_bits(outs[0][3].to(torch.bfloat16), outs[1][3])


def test_linear_dropout_captured_with_device_counter(Q, O, cuda):
    """Forward and backward in one graph: each replay's masks follow the device counter, the same in both."""
    M, nseg, S, K, r = 200, 1, 256, 256, 16
    q, inp, _ = _setup(Q, M, nseg, S, K, r, seed=67, zero_w=True)
    X, dY, A, B = (inp[k].cuda() for k in ("X", "dY", "A", "B"))
    ctr = torch.zeros(1, dtype=torch.int64, device=cuda)
    drop = Q.Dropout(0.5, 8, 50, ctr)

    def step():
        Y = Q.qlora_fused_linear_dropout_fwd(X, q, 1, A, B, 2.0, drop)
        return (Y, *Q.qlora_fused_linear_dropout_bwd(dY, X, q, 1, A, B, 2.0, drop))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = step()
            ctr += 1
    torch.cuda.current_stream().wait_stream(s)
    ctr.zero_()
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        keep = O.dropout_keep(M * K, 0.5, 8, 50 + i).reshape(M, K)
        assert np.array_equal((out[1] != 0).cpu().numpy(), keep)
        plain = Q.Dropout(0.5, 8, 50 + i)
        Y = Q.qlora_fused_linear_dropout_fwd(X, q, 1, A, B, 2.0, plain)
        ref = (Y, *Q.qlora_fused_linear_dropout_bwd(dY, X, q, 1, A, B, 2.0, plain))
        assert all(_same_bits(a, b) for a, b in zip(out, ref)), i


def test_linear_dropout_two_streams(Q, cuda):
    """Independent calls on two streams at once give the bits of the calls one by one."""
    sets = []
    for i in range(2):
        q, inp, _ = _setup(Q, 300, 2, 256, 512, 16, seed=68 + i)
        sets.append((q, inp, Q.Dropout(0.2, i, 5)))
    ref = [_run(Q, q, inp, 2, 2.0, d) for q, inp, d in sets]
    dev = [{k: inp[k].cuda() for k in ("X", "dY", "A", "B")} for _, inp, _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                q, t, d = sets[i][0], dev[i], sets[i][2]
                Y = Q.qlora_fused_linear_dropout_fwd(t["X"], q, 2, t["A"], t["B"], 2.0, d)
                got[i] = (Y, Q.qlora_fused_linear_dropout_bwd(t["dY"], t["X"], q, 2, t["A"], t["B"], 2.0, d))
        torch.cuda.synchronize()
        assert Q.qlora_get_last_error() == 0
        for (Y, g), (rY, rg) in zip(got, ref):
            assert _same_bits(Y, rY) and all(_same_bits(a, b) for a, b in zip(g, rg))


def _ref64(X, W, A, B, s, nseg, mask, dY):
    """The definition in fp64 on the device (large sizes)."""
    S, r = W.shape[0] // nseg, A.shape[0] // nseg
    xd = X * mask
    u = s * xd @ A.T
    Y = X @ W.T
    G = torch.empty(X.shape[0], nseg * r, dtype=torch.float64, device=X.device)
    dB = torch.empty_like(B)
    for i in range(nseg):
        Y[:, i * S:(i + 1) * S] += u[:, i * r:(i + 1) * r] @ B[i * S:(i + 1) * S].T
        G[:, i * r:(i + 1) * r] = s * dY[:, i * S:(i + 1) * S] @ B[i * S:(i + 1) * S]
        dB[i * S:(i + 1) * S] = dY[:, i * S:(i + 1) * S].T @ u[:, i * r:(i + 1) * r]
    return Y, dY @ W + (G @ A) * mask, G.T @ xd, dB


@pytest.mark.parametrize("M,nseg,S,K", [(2048, 3, 4096, 4096), (1531, 1, 4096, 11008)])
def test_linear_dropout_full_size(Q, O, cuda, M, nseg, S, K):
    """LLaMA-7B q/k/v at 2048 tokens and its down projection at a ragged batch."""
    r, s, p = 64, 0.25, 0.05
    q, inp, _ = _setup(Q, M, nseg, S, K, r, seed=69)
    drop = Q.Dropout(p, 17, 1)
    Y, g = _run(Q, q, inp, nseg, s, drop)
    mask = torch.from_numpy(O.dropout_keep(M * K, p, 17, 1).reshape(M, K)).cuda().double()
    t = {k: inp[k].cuda().double() for k in ("X", "dY", "A", "B")}
    ref = _ref64(t["X"], Q.qlora_nf4_dequantize(q).double(), t["A"], t["B"], s * O.dropout_factor(p), nseg, mask, t["dY"])
    for name, got, r64 in zip(("Y", "dX", "dA", "dB"), (Y, *g), ref):
        assert_close_tol(_f64(got), r64.cpu().numpy(), name)
