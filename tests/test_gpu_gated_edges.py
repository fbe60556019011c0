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
