"""Gated feed-forward block at the places where one token class or one value
could go its own way: NaN pre-activations, the borders of the token classes,
and batches of more token tiles than SMs."""
import pytest
import torch

from test_gpu_gated import _dev, _same_bits, _setup

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
