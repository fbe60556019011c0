"""Gated feed-forward block at the places where one token class or one value
could go its own way: NaN pre-activations, the borders of the token classes,
and batches of more token tiles than SMs."""
import pytest
import torch

from test_gpu_gated import _check, _dev, _same_bits, _setup

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu_tanh"]


def _nan_rows(t):
    """(rows all NaN, rows all finite) of a matrix."""
    return torch.isnan(t).all(dim=1), torch.isfinite(t).all(dim=1)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 8, 9, 40, 300])
@pytest.mark.parametrize("half", ["gate", "up"])
def test_nan_pre_activation_reaches_every_gradient_of_it(Q, cuda, act, M, half):
    """One NaN in the kept [g | u].  In g: dG = dH u act'(NaN) and dU = dH act(NaN) are NaN there, so both rows of dB,
    both adapters' dA and the token's dX are; in u: dG alone, so the gate's are and the up adapter's gradients stay
    finite.  No other token's dX and no other row of dB changes."""
    F, K, r = 512, 320, 16
    q, inp, _ = _setup(Q, M, F, K, r, seed=50)
    t = _dev(inp)
    _, GU = Q.qlora_gated_linear_fwd(t["X"], q, t["A"], t["B"], 2.0, act, want_gu=True)
    m0, f0 = M // 2, 77
    bad = GU.clone()
    bad[m0, f0 + (F if half == "up" else 0)] = float("nan")
    ref = Q.qlora_gated_linear_bwd(t["dH"], t["X"], GU, q, t["A"], t["B"], 2.0, act)
    dX, dA, dB = Q.qlora_gated_linear_bwd(t["dH"], t["X"], bad, q, t["A"], t["B"], 2.0, act)
    torch.cuda.synchronize()
    assert Q.qlora_get_last_error() == 0
    tokens = torch.arange(M, device=cuda)
    nan, fin = _nan_rows(dX)
    assert bool(nan[m0]) and _same_bits(dX[tokens != m0], ref[0][tokens != m0])
    nan, fin = _nan_rows(dA)
    both = half == "gate"
    assert bool(nan[:r].all()), "gate adapter's dA"
    assert bool(nan[r:].all() if both else fin[r:].all()), "up adapter's dA"
    nan, fin = _nan_rows(dB)
    hit = torch.zeros(2 * F, dtype=torch.bool, device=cuda)
    hit[f0] = True
    hit[F + f0] = both
    assert torch.equal(nan, hit) and torch.equal(fin, ~hit), "rows of dB"


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 3, 8, 9, 100, 300])
def test_nan_token_gives_a_nan_row_and_no_other(Q, cuda, act, M):
    """A token of NaN through the forward of every token class: its H and GU are NaN, the others keep their bits."""
    q, inp, _ = _setup(Q, M, 512, 320, 16, seed=51)
    t = _dev(inp)
    X = t["X"].clone()
    X[M // 2] = float("nan")
    rows = torch.arange(M, device=cuda) != M // 2
    a = Q.qlora_gated_linear_fwd(t["X"], q, t["A"], t["B"], 2.0, act, want_gu=True)
    b = Q.qlora_gated_linear_fwd(X, q, t["A"], t["B"], 2.0, act, want_gu=True)
    for u, v in zip(a, b):
        assert _same_bits(u[rows], v[rows]) and bool(torch.isnan(v[M // 2]).all())


def _gu64(Q, q, t, s, rows):
    """The pre-activations of the first `rows` tokens from the definition in fp64, U rounded to bf16 as the layer's is."""
    F, r = q.rows // 2, t["B"].shape[1]
    X, A, B = (t[k].double() for k in ("X", "A", "B"))
    U = (s * X[:rows] @ A.T).bfloat16().double()
    Y = X[:rows] @ Q.qlora_nf4_dequantize(q).double().T
    Y[:, :F] += U[:, :r] @ B[:F].T
    Y[:, F:] += U[:, r:] @ B[F:].T
    return Y


@pytest.mark.parametrize("fmt", [dict(), dict(dq=False), dict(blocksize=128, code_type="fp4", dq_type="e4m3")],
                         ids=["nf4", "no_dq", "fp4_128_e4m3"])
@pytest.mark.parametrize("F,K", [(512, 704), (1024, 4096)])
def test_few_tokens_compute_the_same_function_as_many(Q, cuda, F, K, fmt):
    """A call of 8 tokens and the first 8 rows of calls of 9, 100 and 300: the same layer, so the same values up to the
    order of fp32 sums.  Two fp32 sums of K <= 4096 bf16 products in different orders (tensor-core steps of 16 or 64)
    differ by at most (K / 16) 2^-23 = 3e-5 of the sum of magnitudes' root mean square, 1e-4 of H behind the activation
    and the product.  A value then lands on the other side of a rounding border with probability 1e-4 / 2^-7 = 1.3 %,
    where it changes by 2^-7: sqrt(0.013) * 2^-7 = 9e-4 of the norm at most.  (sU is formed by another kernel past 16
    tokens: one more such rounding on the adapter's term, below the base's size; 2e-3 there.)  No value moves by more
    than one bf16 step of the largest of its terms: 2^-7 of the largest |value|."""
    q, inp, _ = _setup(Q, 300, F, K, 16, seed=52, **fmt)
    t = _dev(inp)
    few = Q.qlora_gated_linear_fwd(t["X"][:8], q, t["A"], t["B"], 2.0, want_gu=True)
    for M, tol in ((9, 1e-3), (100, 2e-3), (300, 2e-3)):
        many = Q.qlora_gated_linear_fwd(t["X"][:M], q, t["A"], t["B"], 2.0, want_gu=True)
        for name, a, b in zip(("H", "GU"), few, many):
            a, b = a.double(), b[:8].double()
            assert float((a - b).norm() / b.norm()) <= tol, (name, M)
            assert float((a - b).abs().max()) <= 2.0 ** -7 * float(b.abs().max()), (name, M)
    # against the definition: the output's own rounding, 2^-7 / sqrt(12) = 2.26e-3 of the norm if every value sat at
    # the bottom of its binade (where a rounding weighs most), and the sums' 1e-4
    ref = _gu64(Q, q, t, 2.0, 8)
    assert float((few[1].double() - ref).norm() / ref.norm()) <= 2.4e-3
    H = ref[:, :F] * torch.sigmoid(ref[:, :F]) * ref[:, F:]
    assert float((few[0].double() - H).norm() / H.norm()) <= 2.4e-3
    torch.cuda.synchronize()
    assert Q.qlora_get_last_error() == 0


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 2, 7, 8])
def test_few_tokens_weight_operand_is_the_dequantized_weight(Q, cuda, M, act):
    """Tokens that are unit vectors read the weight back: without an adapter GU is W' itself, bit for bit."""
    F, K = 512, 704
    q, _, _ = _setup(Q, M, F, K, 0, seed=53)
    W = Q.qlora_nf4_dequantize(q)
    for k0 in (0, 17, 255, 256, 640, K - 8):
        X = torch.zeros(M, K, dtype=torch.bfloat16, device=cuda)
        cols = [(k0 + i) % K for i in range(M)]
        X[torch.arange(M), cols] = 1.0
        _, GU = Q.qlora_gated_linear_fwd(X, q, None, None, 1.0, act, want_gu=True)
        assert torch.equal(GU, W[:, cols].T.contiguous()), k0


@pytest.mark.parametrize("M,F,K,r", [
    (8, 768, 448, 24), (9, 768, 448, 24),    # the last size of one kernel and the first of the next, tiles cut
    (128, 768, 448, 24), (128, 1024, 256, 128),  # a full token tile
    (129, 768, 448, 24),
])
@pytest.mark.parametrize("act,p", [("silu", 0.3), ("gelu_tanh", 0.0)])
def test_borders_of_the_token_classes(Q, O, cuda, M, F, K, r, act, p):
    q, inp, Wd = _setup(Q, M, F, K, r, seed=300 + M)
    _check(Q, O, q, inp, Wd, 2.0, act, Q.Dropout(p, 31, 2) if p else None, f"border M={M} F={F} K={K} r={r} {act}")


@pytest.mark.parametrize("M,p", [(9601, 0.2), (19001, 0.0)])
def test_more_token_tiles_than_half_the_sms(Q, O, cuda, M, p):
    """76 and 149 tiles of 128 tokens: the backward's first pass has one column range a tile and writes sG itself."""
    q, inp, Wd = _setup(Q, M, 256, 64, 8, seed=54)
    _check(Q, O, q, inp, Wd, 2.0, "silu", Q.Dropout(p, 8, 3) if p else None, f"M={M}")


@pytest.mark.parametrize("M,F,K,r,p", [(8, 512, 320, 16, 0.0), (200, 768, 448, 24, 0.2), (700, 512, 576, 64, 0.0),
                                       (700, 512, 320, 72, 0.1), (300, 512, 256, 128, 0.0), (9601, 256, 64, 32, 0.0)])
@pytest.mark.parametrize("serial", [False, True])
def test_adapter_gradients_carry_one_rounding(Q, cuda, M, F, K, r, p, serial):
    """dA and dB in fp32 against the gradient at the kept [g | u] in fp64.  dA carries G's rounding to bf16 and dB that
    of dY, one each: a bf16 rounding is uniform over a step of 2^-7 of the value's binade, 2^-7 / sqrt(12) of it, and a
    value's mean square over its binade is 2.16 for the logarithmic distribution of significands: 1.53e-3 of the norm,
    1.7e-3 where large values weigh most.  Two such roundings are 2.2e-3 to 2.4e-3, so the border is 1.95e-3; over
    5000 and more independent roundings the fluctuation is below 2 %.  (M = 8: G has 256 values only, 2.1e-3.)"""
    q, inp, _ = _setup(Q, M, F, K, r, seed=55)
    t = _dev(inp)
    drop = Q.Dropout(p, 3, 7) if p else None
    _, GU = Q.qlora_gated_linear_fwd(t["X"], q, t["A"], t["B"], 2.0, "silu", drop, want_gu=True)
    Q.qlora_debug_inject(6 if serial else 0)
    try:
        dX, dA, dB = Q.qlora_gated_linear_bwd(t["dH"], t["X"], GU, q, t["A"], t["B"], 2.0, "silu", drop)
    finally:
        Q.qlora_debug_inject(0)
    torch.cuda.synchronize()
    assert Q.qlora_get_last_error() == 0
    X, A, B, dH, GU = (x.double() for x in (t["X"], t["A"], t["B"], t["dH"], GU))
    mask = torch.ones_like(X) if drop is None else \
        Q.qlora_dropout(torch.ones(M, K, device=cuda), drop).double().sign()
    s = 2.0 * (1.0 if drop is None else 32768 / (32768 - int(p * 32768 + 0.5)))
    g, u = GU[:, :F], GU[:, F:]
    sig = torch.sigmoid(g)
    dY = torch.cat([dH * u * sig * (1 + g * (1 - sig)), dH * g * sig], dim=1)
    G = s * torch.cat([dY[:, :F] @ B[:F], dY[:, F:] @ B[F:]], dim=1)
    U = s * (X * mask) @ A.T
    rA = G.T @ (X * mask)
    rB = torch.cat([dY[:, :F].T @ U[:, :r], dY[:, F:].T @ U[:, r:]])
    bound = 1.95e-3 if M > 8 else 2.1e-3
    assert float((dA - rA).norm() / rA.norm()) <= bound, "dA"
    assert float((dB - rB).norm() / rB.norm()) <= bound, "dB"


@pytest.mark.parametrize("M", [5, 300])
def test_gradient_values_that_round_to_infinity(Q, cuda, M):
    """dG of 2^127 times 1.999: bf16 rounds it to infinity, and its remainder must not turn the infinity into a NaN:
    sG of that token is infinite, not NaN, so dA's gate columns are infinite where X is not 0."""
    F, K, r = 256, 128, 8
    q, inp, _ = _setup(Q, M, F, K, r, seed=56)
    t = _dev(inp)
    GU = torch.zeros(M, 2 * F, dtype=torch.bfloat16, device=cuda)
    GU[:, :F] = 100.0  # silu'(100) = 1, so dG = dH u
    dH = torch.zeros(M, F, dtype=torch.bfloat16, device=cuda)
    GU[0, F + 3], dH[0, 3] = 2.0 ** 64 * 1.9921875, 2.0 ** 63 * 1.9921875  # product 2^127 * 3.97: over
    B = torch.ones_like(t["B"])
    X = torch.ones_like(t["X"])
    dX, dA, dB = Q.qlora_gated_linear_bwd(dH, X, GU, q, t["A"], B, 1.0)
    torch.cuda.synchronize()
    assert Q.qlora_get_last_error() == 0
    assert bool(torch.isinf(dA[:r]).all())
