"""GPU gated feed-forward block against fp64: H and the kept pre-activations
for every token count class, both activations, with and without adapters and
dropout; the backward from the kept values; a whole training step.

Tolerances: H and GU carry their own bf16 rounding and, in the adapter's term,
that of U; the backward's dY is rounded once to bf16 and reaches dX, G and dB,
which add their own and G's or U's rounding: at most three roundings of 1.7e-3
of the norm each, sqrt(3) * 1.7e-3 = 2.9e-3, below the linear tests' 5e-3.
The largest error of a sum of many rounded terms stays below 1e-2 of the
largest value.  For few tokens the weight's values carry up to 1.6e-3 of bf16
table error, which the activation and the product pass on at most about
threefold (g act'(g) / act(g) <= 1 + |g| / 2 at the values met, u once)."""
import numpy as np
import pytest
import torch

from bit_nf4_quantized_08_b200 import workloads as wl
from conftest import assert_close_tol
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu


def _same_bits(a, b):
    it = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.contiguous().view(it), b.contiguous().view(it))


def _setup(Q, M, F, K, r, seed, dq=True, w_std=None, **fmt):
    # pre-activations of about N(0, 1), as a trained block's
    W = wl.weight(2 * F, K, seed=seed, dtype=torch.bfloat16)
    W = (W.float() * ((w_std or K ** -0.5) / 0.02)).to(torch.bfloat16)
    inp = wl.fused_inputs(M, 2, F, K, max(r, 8), seed=seed, b_std=0.3)
    inp["dH"] = inp.pop("dY")[:, :F].contiguous()
    if r == 0:
        inp["A"] = inp["B"] = None
    q = Q.qlora_nf4_quantize(W.cuda(), double_quant=dq, **fmt)
    return q, inp, wl.bits(Q.qlora_nf4_dequantize(q).cpu())


def _dev(inp):
    return {k: None if v is None else v.cuda() for k, v in inp.items()}


def _bits_or_zero(t, shape):
    return np.zeros(shape, np.uint16) if t is None else wl.bits(t)


def _np(t):
    return t.double().cpu().numpy()


def _check(Q, O, q, inp, Wd, s, act, drop, tag, grad_dtype=torch.float32, want_dx=True):
    t = _dev(inp)
    H, GU = Q.qlora_gated_linear_fwd(t["X"], q, t["A"], t["B"], s, act, drop, want_gu=True)
    H2, none = Q.qlora_gated_linear_fwd(t["X"], q, t["A"], t["B"], s, act, drop)
    g = Q.qlora_gated_linear_bwd(t["dH"], t["X"], GU, q, t["A"], t["B"], s, act, drop, want_dx=want_dx,
                                 grad_dtype=grad_dtype)
    torch.cuda.synchronize()
    assert Q.qlora_get_last_error() == 0
    assert none is None and _same_bits(H, H2), f"{tag}: H depends on whether GU is kept"
    N, K = Wd.shape
    bits = (wl.bits(inp["X"]), Wd, _bits_or_zero(inp["A"], (16, K)), _bits_or_zero(inp["B"], (N, 8)))
    d = None if drop is None else (drop.p, drop.seed, drop.offset)
    rH, rGU = O.gated_fwd(*bits, s, act, d)
    assert_close_tol(_np(H), rH, f"H {tag}")
    assert_close_tol(_np(GU), rGU, f"GU {tag}")
    # the backward is a function of the kept (rounded) GU
    ref = O.gated_bwd(wl.bits(inp["dH"]), bits[0], wl.bits(GU.cpu()), *bits[1:], s, act, d)
    for name, got, r in zip(("dX", "dA", "dB"), g, ref):
        if got is not None:
            assert_close_tol(_np(got), r, f"{name} {tag}")
    return H, GU, g


CASES = [
    # M, F, K, r: one token, every small-token kernel and its borders, ragged token tiles, several column tiles
    (1, 256, 64, 8), (2, 512, 128, 16), (15, 256, 320, 64), (16, 768, 448, 24), (17, 256, 192, 8), (31, 512, 256, 40),
    (33, 256, 512, 128), (64, 1024, 256, 64), (65, 256, 64, 8), (129, 512, 320, 16), (300, 256, 512, 32),
    (513, 768, 576, 64), (1100, 512, 192, 128),
]


@pytest.mark.parametrize("M,F,K,r", CASES)
@pytest.mark.parametrize("act,p", [("silu", 0.3), ("gelu_tanh", 0.0)])
def test_gated_parity(Q, O, cuda, M, F, K, r, act, p):
    q, inp, Wd = _setup(Q, M, F, K, r, seed=100 + M)
    drop = Q.Dropout(p, 31, 2) if p else None
    _check(Q, O, q, inp, Wd, 2.0, act, drop, f"M={M} F={F} K={K} r={r} {act}",
           torch.bfloat16 if M % 2 else torch.float32)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gated_without_adapter(Q, O, cuda, M):
    q, inp, Wd = _setup(Q, M, 512, 320, 0, seed=7)
    _, _, g = _check(Q, O, q, inp, Wd, 1.0, "silu", None, f"r=0 M={M}")
    assert g[1] is None and g[2] is None
    # a dropout without an adapter drops nothing
    t = _dev(inp)
    H, _ = Q.qlora_gated_linear_fwd(t["X"], q, None, None, 1.0, "silu", Q.Dropout(0.5, 1))
    assert _same_bits(H, Q.qlora_gated_linear_fwd(t["X"], q, None, None, 1.0, "silu")[0])


@pytest.mark.parametrize("fmt", [dict(dq=False), dict(blocksize=128, code_type="fp4"), dict(blocksize=256, dq_type="e4m3")],
                         ids=["no_dq", "fp4_128", "e4m3_256"])
@pytest.mark.parametrize("M", [6, 50, 200])
def test_gated_formats(Q, O, cuda, fmt, M):
    q, inp, Wd = _setup(Q, M, 512, 512, 16, seed=8, **fmt)
    _check(Q, O, q, inp, Wd, 2.0, "silu", Q.Dropout(0.1, 1, 1), f"{fmt} M={M}")


@pytest.mark.parametrize("mode", [2, 3, 4, 6, 7, 8], ids=["streamk7", "single_cta_grid", "pair_streamk4", "serial_bwd",
                                                          "warp_mma", "tcgen05_small"])
@pytest.mark.parametrize("M", [10, 30, 600])
def test_gated_alternate_schedules(Q, O, cuda, mode, M):
    q, inp, Wd = _setup(Q, M, 512, 512, 16, seed=9)
    Q.qlora_debug_inject(mode)
    try:
        _check(Q, O, q, inp, Wd, 2.0, "silu", Q.Dropout(0.1, 4, 4), f"mode {mode} M={M}")
    finally:
        Q.qlora_debug_inject(0)


@pytest.mark.parametrize("M", [4, 20, 200])
def test_gated_saturated_activations(Q, O, cuda, M):
    """Pre-activations of a few hundred: exp overflows and vanishes, H and the gradients stay finite and right."""
    for act in ("silu", "gelu_tanh"):
        q, inp, Wd = _setup(Q, M, 256, 256, 8, seed=10, w_std=10.0)
        with np.errstate(over="ignore"):
            _check(Q, O, q, inp, Wd, 1.0, act, None, f"saturated {act} M={M}")


@pytest.mark.parametrize("M", [3, 24, 70, 333])
def test_gated_guards_and_repeat(Q, cuda, M):
    F, K, r = 512, 320, 24
    q, inp, _ = _setup(Q, M, F, K, r, seed=11)
    t = _dev(inp)
    drop = Q.Dropout(0.15, 2, 2)
    outs = []
    for _ in range(2):
        G = {"H": Guarded((M, F), torch.bfloat16), "GU": Guarded((M, 2 * F), torch.bfloat16),
             "dX": Guarded((M, K), torch.bfloat16), "dA": Guarded((2 * r, K), torch.float32),
             "dB": Guarded((2 * F, r), torch.float32),
             "wf": Guarded((Q.qlora_gated_linear_workspace(M, q, r, False),), torch.uint8),
             "wb": Guarded((Q.qlora_gated_linear_workspace(M, q, r, True),), torch.uint8)}
        Q.qlora_gated_linear_fwd(t["X"], q, t["A"], t["B"], 2.0, "silu", drop, H=G["H"].t, GU=G["GU"].t, ws=G["wf"].t)
        Q.qlora_gated_linear_bwd(t["dH"], t["X"], G["GU"].t, q, t["A"], t["B"], 2.0, "silu", drop, dX=G["dX"].t,
                                 dA=G["dA"].t, dB=G["dB"].t, ws=G["wb"].t)
        torch.cuda.synchronize()
        assert Q.qlora_get_last_error() == 0
        for k, g in G.items():
            g.check(k)
        outs.append([G[k].t.clone() for k in ("H", "GU", "dX", "dA", "dB")])
    assert all(_same_bits(a, b) for a, b in zip(*outs))


def test_gated_empty_batch_and_refusals(Q, cuda):
    q, inp, _ = _setup(Q, 4, 256, 128, 8, seed=12)
    t = _dev(inp)
    X = torch.empty(0, 128, dtype=torch.bfloat16, device=cuda)
    H, GU = Q.qlora_gated_linear_fwd(X, q, t["A"], t["B"], 1.0, want_gu=True)
    assert H.shape == (0, 256) and GU.shape == (0, 512)
    dA = torch.ones(16, 128, device=cuda)
    dX, dA, dB = Q.qlora_gated_linear_bwd(H, X, GU, q, t["A"], t["B"], 1.0, dA=dA)
    torch.cuda.synchronize()
    assert not dA.any() and not dB.any()
    with pytest.raises(ValueError):
        Q.qlora_gated_linear_fwd(t["X"], q, t["A"], t["B"], 1.0, act="relu")
    with pytest.raises(ValueError):
        Q.qlora_gated_linear_fwd(t["X"][:, ::2], q, t["A"], t["B"], 1.0)
    with pytest.raises(Q.QloraError) as e:
        Q.qlora_gated_linear_fwd(t["X"], q, t["A"], t["B"], 1.0, dropout=Q.Dropout(1.0, 1))
    assert e.value.status == Q.QLORA_ERR_INVALID_ARG


def test_gated_graph_and_shared_workspace(Q, cuda):
    """Two captured graphs that share one workspace, replayed in turn, and eager calls between."""
    sets = []
    for i, M in enumerate((5, 300)):
        q, inp, _ = _setup(Q, M, 512, 256, 16, seed=13 + i)
        sets.append((q, _dev(inp), Q.Dropout(0.2, i, 1)))
    need = max(Q.qlora_gated_linear_workspace(t["X"].shape[0], q, 16, b) for q, t, _ in sets for b in (False, True))
    ws = torch.empty(need, dtype=torch.uint8, device=cuda)

    def step(q, t, d):
        H, GU = Q.qlora_gated_linear_fwd(t["X"], q, t["A"], t["B"], 2.0, "silu", d, want_gu=True, ws=ws)
        return (H, GU, *Q.qlora_gated_linear_bwd(t["dH"], t["X"], GU, q, t["A"], t["B"], 2.0, "silu", d, ws=ws))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(s):
        ref = [[x.clone() for x in step(*a)] for a in sets]
        for a in sets:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(step(*a))
            graphs.append(g)
        for i in (0, 1, 1, 0, 1):
            for o in outs[i]:
                o.fill_(0)
            graphs[i].replay()
            step(*sets[1 - i])
            s.synchronize()
            assert all(_same_bits(a, b) for a, b in zip(outs[i], ref[i])), i
    assert Q.qlora_get_last_error() == 0


@pytest.mark.parametrize("M,F,K", [(1, 11008, 4096), (16, 11008, 4096), (48, 11008, 4096), (2048, 11008, 4096),
                                   (777, 22016, 8192)])
def test_gated_full_size(Q, O, cuda, M, F, K):
    """LLaMA-7B (all token classes) and LLaMA-65B gate/up, fp64 on the device."""
    r, s, p = 64, 0.25, 0.05
    q, inp, _ = _setup(Q, M, F, K, r, seed=14, w_std=0.02)
    t = _dev(inp)
    drop = Q.Dropout(p, 5, 5)
    H, GU = Q.qlora_gated_linear_fwd(t["X"], q, t["A"], t["B"], s, "silu", drop, want_gu=True)
    dX, dA, dB = Q.qlora_gated_linear_bwd(t["dH"], t["X"], GU, q, t["A"], t["B"], s, "silu", drop)
    torch.cuda.synchronize()
    assert Q.qlora_get_last_error() == 0
    mask = torch.from_numpy(O.dropout_keep(M * K, p, 5, 5).reshape(M, K)).cuda().double()
    W = Q.qlora_nf4_dequantize(q).double()
    X, A, B, dH = (t[k].double() for k in ("X", "A", "B", "dH"))
    s1 = s * O.dropout_factor(p)
    xd = X * mask
    u = s1 * xd @ A.T
    Y = X @ W.T
    Y[:, :F] += u[:, :r] @ B[:F].T
    Y[:, F:] += u[:, r:] @ B[F:].T
    assert_close_tol(_np(GU), Y.cpu().numpy(), "GU")
    sig = torch.sigmoid(Y[:, :F])
    assert_close_tol(_np(H), (Y[:, :F] * sig * Y[:, F:]).cpu().numpy(), "H")
    g, up = GU[:, :F].double(), GU[:, F:].double()
    sig = torch.sigmoid(g)
    dY = torch.cat([dH * up * sig * (1 + g * (1 - sig)), dH * g * sig], dim=1)
    G = s1 * torch.cat([dY[:, :F] @ B[:F], dY[:, F:] @ B[F:]], dim=1)
    assert_close_tol(_np(dX), (dY @ W + (G @ A) * mask).cpu().numpy(), "dX")
    assert_close_tol(_np(dA), (G.T @ xd).cpu().numpy(), "dA")
    assert_close_tol(_np(dB), torch.cat([dY[:, :F].T @ u[:, :r], dY[:, F:].T @ u[:, r:]]).cpu().numpy(), "dB")


def test_feed_forward_training_step(Q, O, cuda):
    """The operators as a step uses them: gate/up with dropout, the down projection with its own, residual dropout,
    the backward of all three, and the adapters' optimizer step; each against fp64 on what the one before gave."""
    M, F, K, r, s = 260, 512, 256, 16, 2.0
    q1, inp, W1 = _setup(Q, M, F, K, r, seed=15)
    t = _dev(inp)
    Wdn = wl.weight(K, F, seed=16, dtype=torch.bfloat16)
    q2 = Q.qlora_nf4_quantize(Wdn.cuda())
    W2 = wl.bits(Q.qlora_nf4_dequantize(q2).cpu())
    i2 = wl.linear_inputs(M, K, F, r, seed=17)
    A2, B2, dO = i2["A"].cuda(), (i2["B"].float() * 30).to(torch.bfloat16).cuda(), i2["dY"].cuda()
    d1, d2, d3 = Q.Dropout(0.1, 40, 0), Q.Dropout(0.1, 40, 1), Q.Dropout(0.2, 40, 2)
    H, GU = Q.qlora_gated_linear_fwd(t["X"], q1, t["A"], t["B"], s, "silu", d1, want_gu=True)
    Yd = Q.qlora_fused_linear_dropout_fwd(H, q2, 1, A2, B2, s, d2)
    out = Q.qlora_dropout(Yd, d3)
    dYd = Q.qlora_dropout(dO, d3)
    dH, dA2, dB2 = Q.qlora_fused_linear_dropout_bwd(dYd, H, q2, 1, A2, B2, s, d2)
    dX, dA1, dB1 = Q.qlora_gated_linear_bwd(dH, t["X"], GU, q1, t["A"], t["B"], s, "silu", d1)
    flat_g = torch.cat([x.reshape(-1) for x in (dA1, dB1, dA2, dB2)])
    p = torch.cat([x.float().reshape(-1) for x in (t["A"], t["B"], A2, B2)])
    m, v, pb, p0 = torch.zeros_like(p), torch.zeros_like(p), torch.empty_like(p, dtype=torch.bfloat16), p.cpu().double().numpy()
    Q.qlora_adamw_step(p, m, v, flat_g, pb, lr=1e-3, step=1)
    torch.cuda.synchronize()
    assert Q.qlora_get_last_error() == 0
    b = lambda x: wl.bits(x.cpu())
    rH, _ = O.gated_fwd(b(t["X"]), W1, b(t["A"]), b(t["B"]), s, "silu", (0.1, 40, 0))
    assert_close_tol(_np(H), rH, "H")
    assert_close_tol(_np(Yd), O.dropout_linear_fwd(b(H), W2, b(A2), b(B2), s, 1, (0.1, 40, 1)), "down")
    keep = O.dropout_keep(M * K, 0.2, 40, 2).reshape(M, K)
    assert np.array_equal(_np(out) != 0, keep & (_np(Yd) != 0))
    assert np.array_equal(_np(dYd) != 0, keep & (_np(dO) != 0))
    for got, ref in zip((dH, dA2, dB2), O.dropout_linear_bwd(_np(dYd), b(H), W2, b(A2), b(B2), s, 1, (0.1, 40, 1))):
        assert_close_tol(_np(got), ref, "down backward")
    for got, ref in zip((dX, dA1, dB1), O.gated_bwd(b(dH), b(t["X"]), b(GU), W1, b(t["A"]), b(t["B"]), s, "silu",
                                                    (0.1, 40, 0))):
        assert_close_tol(_np(got), ref, "gate/up backward")
    # the first AdamW step moves every parameter against its gradient by lr (up to eps)
    g = flat_g.cpu().double().numpy()
    big = np.abs(g) > 1e-4
    step = _np(p) - p0
    assert np.max(np.abs(step[big] + 1e-3 * np.sign(g[big]))) <= 1e-3 * 1e-3 + 2.0 ** -23 * np.max(np.abs(p0))


@pytest.mark.parametrize("M", [30, 300])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_gated_backward_without_dx(Q, O, cuda, M, p):
    """dA and dB alone (the first layer of a model): the bits of the whole backward's."""
    q, inp, Wd = _setup(Q, M, 512, 320, 24, seed=18)
    drop = Q.Dropout(p, 3, 1) if p else None
    _, GU, g = _check(Q, O, q, inp, Wd, 2.0, "silu", drop, f"no dX M={M}", want_dx=False)
    assert g[0] is None
    t = _dev(inp)
    Q.qlora_debug_inject(6)  # the same GEMM split (serial order), with dX
    try:
        full = Q.qlora_gated_linear_bwd(t["dH"], t["X"], GU, q, t["A"], t["B"], 2.0, "silu", drop)
    finally:
        Q.qlora_debug_inject(0)
    torch.cuda.synchronize()
    assert _same_bits(g[1], full[1]) and _same_bits(g[2], full[2])


def test_gated_backward_in_a_capture_of_its_own(Q, cuda):
    """Forward and backward captured and replayed on another stream than their inputs', twice, give the eager bits."""
    M = 200
    q, inp, _ = _setup(Q, M, 512, 256, 16, seed=19)
    t = _dev(inp)
    d = Q.Dropout(0.1, 2, 9)

    def step():
        H, GU = Q.qlora_gated_linear_fwd(t["X"], q, t["A"], t["B"], 2.0, "silu", d, want_gu=True)
        return (H, GU, *Q.qlora_gated_linear_bwd(t["dH"], t["X"], GU, q, t["A"], t["B"], 2.0, "silu", d))

    ref = [x.clone() for x in step()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = step()
    for _ in range(2):
        for o in out:
            o.fill_(0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        assert Q.qlora_get_last_error() == 0
        assert all(_same_bits(a, b) for a, b in zip(out, ref))


def test_waits_run_out_and_recover(Q, cuda):
    """Without their producers' loads every kernel of the gated and dropout calls gives up after the bound, records
    the timeout and returns; the next calls are right."""
    sets = []
    for M in (5, 100, 300):
        q, inp, _ = _setup(Q, M, 512, 512, 16, seed=20)
        sets.append((q, _dev(inp)))
    d = Q.Dropout(0.2, 1, 1)

    def calls(q, t):
        H, GU = Q.qlora_gated_linear_fwd(t["X"], q, t["A"], t["B"], 2.0, "silu", d, want_gu=True)
        g = Q.qlora_gated_linear_bwd(t["dH"], t["X"], GU, q, t["A"], t["B"], 2.0, "silu", d)
        Y = Q.qlora_fused_linear_dropout_fwd(t["X"], q, 2, t["A"], t["B"], 2.0, d)
        b = Q.qlora_fused_linear_dropout_bwd(Y, t["X"], q, 2, t["A"], t["B"], 2.0, d)
        torch.cuda.synchronize()
        return (H, GU, *g, Y, *b)

    ref = [calls(*a) for a in sets]
    assert Q.qlora_get_last_error() == 0
    Q.qlora_set_wait_timeout_ns(5_000_000)
    Q.qlora_debug_inject(1)
    try:
        for a in sets:
            calls(*a)
            assert Q.qlora_get_last_error() == Q.QLORA_ERR_TIMEOUT
    finally:
        Q.qlora_debug_inject(0)
        Q.qlora_set_wait_timeout_ns(0)
    for a, r in zip(sets, ref):
        got = calls(*a)
        assert Q.qlora_get_last_error() == 0
        assert all(_same_bits(x, y) for x, y in zip(got, r))


def test_workspace_of_another_place_is_refused(Q, cuda):
    """A workspace on another device, or with gaps, would be written out of its bounds."""
    q, inp, _ = _setup(Q, 8, 256, 128, 8, seed=19)
    t = _dev(inp)
    n = Q.qlora_gated_linear_workspace(8, q, 8, True) + Q.qlora_gated_linear_workspace(8, q, 8, False)
    bad = [torch.empty(n, dtype=torch.uint8), torch.empty(2 * n, dtype=torch.uint8, device=cuda)[::2]]
    dY = torch.zeros(8, 512, dtype=torch.bfloat16, device=cuda)
    for ws in bad:
        for call in (lambda: Q.qlora_gated_linear_fwd(t["X"], q, t["A"], t["B"], 1.0, ws=ws),
                     lambda: Q.qlora_gated_linear_bwd(t["dH"], t["X"], dY, q, t["A"], t["B"], 1.0, ws=ws),
                     lambda: Q.qlora_fused_linear_dropout_fwd(t["X"], q, 2, t["A"], t["B"], 1.0, None, ws=ws),
                     lambda: Q.qlora_fused_linear_dropout_bwd(dY, t["X"], q, 2, t["A"], t["B"], 1.0, None, ws=ws)):
            with pytest.raises(ValueError, match="ws must be"):
                call()


def test_gated_calls_on_several_streams_at_once(Q, cuda):
    """Forward and backward of three token classes on a stream each, with a workspace each: the bits of calls alone."""
    sets = []
    for M in (7, 100, 400):
        q, inp, _ = _setup(Q, M, 1024, 512, 16, seed=30 + M)
        sets.append((q, _dev(inp), Q.Dropout(0.2, M, 1)))

    def calls(q, t, d):
        H, GU = Q.qlora_gated_linear_fwd(t["X"], q, t["A"], t["B"], 2.0, "silu", d, want_gu=True)
        return (H, GU, *Q.qlora_gated_linear_bwd(t["dH"], t["X"], GU, q, t["A"], t["B"], 2.0, "silu", d))

    ref = [calls(*a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(5):
        for a, s in zip(sets, streams):
            with torch.cuda.stream(s):
                got.append(calls(*a))
    torch.cuda.synchronize()
    assert Q.qlora_get_last_error() == 0
    for i, g in enumerate(got):
        assert all(_same_bits(a, b) for a, b in zip(g, ref[i % len(sets)]))


@pytest.mark.parametrize("M", [9, 48, 200])
def test_gated_token_of_nan_stays_in_its_row(Q, cuda, M):
    """A token of NaN (an unused slot of a padded batch) changes no other token's H, GU or dX."""
    q, inp, _ = _setup(Q, M, 512, 320, 16, seed=33)
    t = _dev(inp)
    bad = M // 2
    rows = torch.arange(M, device=cuda) != bad
    X2, dH2 = t["X"].clone(), t["dH"].clone()
    X2[bad] = float("nan")
    dH2[bad] = float("nan")
    d = Q.Dropout(0.2, 3, 1)
    outs = []
    for X, dH in ((t["X"], t["dH"]), (X2, dH2)):
        H, GU = Q.qlora_gated_linear_fwd(X, q, t["A"], t["B"], 2.0, "silu", d, want_gu=True)
        dX, _, _ = Q.qlora_gated_linear_bwd(dH, X, GU, q, t["A"], t["B"], 2.0, "silu", d)
        outs.append((H, GU, dX))
    torch.cuda.synchronize()
    assert Q.qlora_get_last_error() == 0
    for a, b in zip(*outs):
        assert _same_bits(a[rows], b[rows]) and torch.isnan(b[bad]).all()


@pytest.mark.parametrize("F,K,r", [
    (256, 256, 8),     # one unit column, every warp on it
    (512, 704, 72),    # two unit columns and three blocks after them, adapters ending inside a k-step
    (768, 2240, 128),  # eight unit columns, two warps each
    (256, 4416, 24),   # seventeen: a warp has two of them
    (9728, 576, 16),   # more hidden columns an SM than fit one reduction
    (512, 128, 0),     # no whole unit, no adapter
])
@pytest.mark.parametrize("M", [1, 5, 8])
def test_gated_few_tokens(Q, O, cuda, M, F, K, r):
    q, inp, Wd = _setup(Q, M, F, K, r, seed=200 + M)
    drop = Q.Dropout(0.2, 5, M) if r and M == 5 else None
    _check(Q, O, q, inp, Wd, 2.0, "gelu_tanh" if M == 8 else "silu", drop, f"few M={M} F={F} K={K} r={r}")


@pytest.mark.parametrize("M", [1, 8, 12])
def test_gated_few_tokens_captured(Q, cuda, M):
    """A captured decoding call replayed on new inputs, after calls of other sizes in the same workspace."""
    q, inp, _ = _setup(Q, M, 1024, 512, 16, seed=41)
    t = _dev(inp)
    ws = torch.full((Q.qlora_gated_linear_workspace(128, q, 16, False),), 0xFF, dtype=torch.uint8, device=cuda)
    X = t["X"].clone()
    H = torch.empty(M, 1024, dtype=torch.bfloat16, device=cuda)

    def call(x, out):
        return Q.qlora_gated_linear_fwd(x, q, t["A"], t["B"], 2.0, H=out, ws=ws)[0]

    call(X, H)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        call(X, H)
    for i in range(3):
        X.copy_(t["X"] * (i + 1))
        Q.qlora_gated_linear_fwd(t["X"].repeat(40 // M + 1, 1), q, t["A"], t["B"], 2.0, ws=ws)
        g.replay()
        assert _same_bits(H, call(X, torch.empty_like(H))), i
    torch.cuda.synchronize()
    assert Q.qlora_get_last_error() == 0


def test_gated_without_workspace(Q, cuda):
    """Up to 8 tokens without an adapter need no workspace: the query gives 0 and the call takes NULL."""
    import ctypes

    from bit_nf4_quantized_08_b200 import _lib
    q, inp, _ = _setup(Q, 8, 256, 320, 0, seed=42)
    X = inp["X"].cuda()
    assert Q.qlora_gated_linear_workspace(8, q, 0, False) == 0
    H = torch.empty(8, 256, dtype=torch.bfloat16, device=cuda)
    st = _lib.lib().qlora_gated_linear_fwd(X.data_ptr(), 8, ctypes.byref(q.c_struct()), None, None, 0, 1.0, 0, None,
                                           H.data_ptr(), None, None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert _same_bits(H, Q.qlora_gated_linear_fwd(X, q, None, None, 1.0)[0])
