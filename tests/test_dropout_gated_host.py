"""Dropout and gated feed-forward without a GPU: the generator's published
known answers, the mask's statistics, the oracle's gradients against
differences and autograd, and the entry points' refusals."""
import ctypes

import numpy as np
import pytest
import torch

from bit_nf4_quantized_08_b200 import workloads as wl

FAKE = 0x7F0000000000  # 256-byte aligned stand-in pointer; never dereferenced


def test_philox_known_answers(O):
    """The generator's authors' known-answer vectors of Philox-4x32-10."""
    ones = 0xFFFFFFFF
    assert O.philox4x32((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert O.philox4x32((ones,) * 4, (ones,) * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert O.philox4x32((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_keep_mask_is_the_definition(O):
    """The vectorised mask against single Philox blocks, past 2^32 blocks too."""
    p, seed, off = 0.3, 0x0123456789ABCDEF, 0xFEDCBA9876543210
    T = O.dropout_threshold(p)
    for first in (0, 8 * 41, 8 * ((1 << 32) + 3)):
        got = O.dropout_keep(21, p, seed, off, first)
        for i in range(21):
            blk, j = divmod(first + i, 8)
            w = O.philox4x32((blk & 0xFFFFFFFF, blk >> 32, off & 0xFFFFFFFF, off >> 32),
                             (seed & 0xFFFFFFFF, seed >> 32))[j >> 1]
            assert got[i] == (((w >> (16 * (j & 1))) & 0x7FFF) >= T)


@pytest.mark.parametrize("p", [0.05, 0.1, 0.5, 0.9])
def test_keep_rate_and_factor(O, p):
    """Rate within six standard deviations of 1 - T/2^15; factor its inverse."""
    n = 1 << 20
    keep = O.dropout_keep(n, p, 7, 1)
    q = 1 - O.dropout_threshold(p) / 32768
    assert abs(keep.mean() - q) <= 6 * np.sqrt(q * (1 - q) / n)
    assert O.dropout_factor(p) == 1 / q
    other = O.dropout_keep(n, p, 7, 2)
    both = (keep & other).mean()
    assert abs(both - q * q) <= 6 * np.sqrt(q * q * (1 - q * q) / n)


def _small(seed, M=9, nseg=2, S=24, K=16, r=8):
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    return mk(M, K), mk(nseg * S, K), mk(nseg * r, K), mk(nseg * S, r), mk(M, nseg * S), mk(M, S)


@pytest.mark.parametrize("drop", [None, (0.4, 11, 5)], ids=["p0", "p0.4"])
def test_oracle_dropout_linear_vs_autograd(O, drop):
    X, W, A, B, dY, _ = _small(1)
    s, nseg, r = 0.5, 2, 8
    x, a, b = (t.double().requires_grad_() for t in (X, A, B))
    mask = torch.ones_like(x) if drop is None else \
        torch.from_numpy(O.dropout_keep(x.numel(), *drop).reshape(x.shape).astype(np.float64)) * O.dropout_factor(drop[0])
    u = s * (x * mask) @ a.T
    y = x @ W.double().T + torch.cat([u[:, i * r:(i + 1) * r] @ b[i * 24:(i + 1) * 24].T for i in range(nseg)], dim=1)
    y.backward(dY.double())
    bits = [wl.bits(t) for t in (X, W, A, B)]
    np.testing.assert_allclose(O.dropout_linear_fwd(*bits, s, nseg, drop), y.detach().numpy(), rtol=1e-12, atol=1e-12)
    for got, ref in zip(O.dropout_linear_bwd(dY.double().numpy(), *bits, s, nseg, drop), (x.grad, a.grad, b.grad)):
        np.testing.assert_allclose(got, ref.numpy(), rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_oracle_act_gradient_vs_differences(O, act):
    g = np.linspace(-12, 12, 4001)
    h = 1e-5
    v, d = O.gated_act(act, g)
    num = (O.gated_act(act, g + h)[0] - O.gated_act(act, g - h)[0]) / (2 * h)
    # central differences: truncation h^2 |f'''| / 6 < 1e-10, rounding |f| 2^-53 / h < 2e-10
    assert np.max(np.abs(num - d)) < 1e-9
    ref = {"silu": torch.nn.functional.silu, "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}
    np.testing.assert_allclose(v, ref[act](torch.from_numpy(g)).numpy(), rtol=1e-11, atol=1e-14)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_oracle_gated_gradient_vs_differences(O, act):
    """d<H, C>/dtheta by central differences along a random direction of X, A and B."""
    X, W, A, B, _, dH = _small(3)
    W = (W.float() * 0.2).to(torch.bfloat16)
    s, drop = 0.5, (0.25, 9, 2)
    xf, wf, af, bf = (t.double().numpy() for t in (X, W, A, B))
    mask = O.dropout_keep(xf.size, *drop).reshape(xf.shape) * O.dropout_factor(drop[0])

    def loss(x, a, b):
        u = s * (x * mask) @ a.T
        y = x @ wf.T + np.concatenate([u[:, :8] @ b[:24].T, u[:, 8:] @ b[24:].T], axis=1)
        return np.sum(O.gated_act(act, y[:, :24])[0] * y[:, 24:] * dH.double().numpy()), y

    _, y = loss(xf, af, bf)
    # the backward reads GU as bf16: feed it fp64 values through the oracle's parts
    v, d = O.gated_act(act, y[:, :24])
    dh = dH.double().numpy()
    dY = np.concatenate([dh * y[:, 24:] * d, dh * v], axis=1)
    grads = O.dropout_linear_bwd(dY, wl.bits(X), wl.bits(W), wl.bits(A), wl.bits(B), s, 2, drop)
    rng = np.random.default_rng(0)
    for i, t in enumerate((xf, af, bf)):
        e = rng.normal(size=t.shape)
        h = 1e-6
        args = [xf, af, bf]
        hi = loss(*[q + h * e if j == i else q for j, q in enumerate(args)])[0]
        lo = loss(*[q - h * e if j == i else q for j, q in enumerate(args)])[0]
        ref = float(np.sum(grads[i] * e))
        assert abs((hi - lo) / (2 * h) - ref) <= 1e-6 * (abs(ref) + np.linalg.norm(grads[i])), i


# --------------------------------------------------------------------------- refusals
def _w(rows=512, cols=256, **kw):
    from bit_nf4_quantized_08_b200._lib import CNF4Weight
    f = dict(blocksize=64, dq=1, codes=FAKE)
    f.update(kw)
    return CNF4Weight(rows, cols, f["blocksize"], f["dq"], f["codes"], FAKE, FAKE, FAKE, FAKE, 0, 0)


def _cfg(p=0.1, seed=1, offset=0, dev=None):
    from bit_nf4_quantized_08_b200._lib import CDropoutConfig
    return ctypes.byref(CDropoutConfig(p, seed, offset, dev))


BAD_DROPOUT = [float("nan"), -0.1, 1.0, 1.5, float("inf"), 1 - 2.0 ** -17]


def test_dropout_rejects(Q):
    from bit_nf4_quantized_08_b200._lib import lib, QLORA_BF16, QLORA_F32, QLORA_ERR_INVALID_ARG as BAD
    f = lib().qlora_dropout
    for p in BAD_DROPOUT:
        assert f(FAKE, QLORA_BF16, 64, _cfg(p), FAKE, None) == BAD
    assert f(FAKE, QLORA_BF16, 64, None, FAKE, None) == BAD
    assert f(FAKE, 2, 64, _cfg(), FAKE, None) == BAD
    assert f(FAKE, QLORA_F32, -1, _cfg(), FAKE, None) == BAD
    assert f(None, QLORA_F32, 64, _cfg(), FAKE, None) == BAD
    assert f(FAKE, QLORA_F32, 64, _cfg(), None, None) == BAD
    assert f(FAKE + 4, QLORA_F32, 64, _cfg(), FAKE, None) == BAD
    assert f(FAKE, QLORA_BF16, 64, _cfg(), FAKE + 2, None) == BAD
    assert f(FAKE, QLORA_BF16, 64, _cfg(dev=FAKE + 4), FAKE, None) == BAD
    assert f(None, QLORA_BF16, 0, _cfg(), None, None) == 0


def test_linear_dropout_rejects(Q):
    from bit_nf4_quantized_08_b200._lib import lib, QLORA_ERR_INVALID_ARG as BAD, QLORA_ERR_UNSUPPORTED as UNS
    big, L = 1 << 36, lib()
    f, b = L.qlora_fused_linear_dropout_fwd, L.qlora_fused_linear_dropout_bwd
    w = ctypes.byref(_w())

    def fwd(X=FAKE, M=16, w=w, nseg=2, A=FAKE, B=FAKE, r=8, drop=_cfg(), Y=FAKE, ws=FAKE, n=big):
        return f(X, M, w, nseg, A, B, r, 1.0, drop, Y, ws, n, None)

    def bwd(dY=FAKE, X=FAKE, M=16, w=w, nseg=2, A=FAKE, B=FAKE, r=8, drop=_cfg(), dX=FAKE, gd=0, dA=FAKE, dB=FAKE,
            ws=FAKE, n=big):
        return b(dY, X, M, w, nseg, A, B, r, 1.0, drop, dX, gd, dA, dB, ws, n, None)

    for p in BAD_DROPOUT:
        assert fwd(drop=_cfg(p)) == BAD and bwd(drop=_cfg(p)) == BAD
    assert fwd(w=ctypes.byref(_w(512, 200))) == UNS and bwd(w=ctypes.byref(_w(512, 200))) == UNS
    assert fwd(w=ctypes.byref(_w(400, 256))) == UNS       # segments not whole tiles
    assert fwd(r=12) == UNS and fwd(r=136) == UNS and fwd(r=-8) == BAD and fwd(nseg=0) == BAD
    assert fwd(X=None) == BAD and fwd(Y=FAKE + 2) == BAD and fwd(A=None) == BAD and fwd(B=FAKE + 8) == BAD
    assert fwd(n=1024) == BAD and fwd(ws=None) == BAD and fwd(ws=FAKE + 8) == BAD and fwd(M=-1) == BAD
    assert fwd(w=None) == BAD and fwd(M=0, X=None, Y=None) == 0
    assert bwd(gd=2) == BAD and bwd(dA=None) == BAD and bwd(dB=FAKE + 4) == BAD and bwd(dX=FAKE + 2) == BAD
    assert bwd(dY=None) == BAD and bwd(X=None) == BAD and bwd(n=1024) == BAD


def test_gated_rejects(Q):
    from bit_nf4_quantized_08_b200._lib import lib, QLORA_ERR_INVALID_ARG as BAD, QLORA_ERR_UNSUPPORTED as UNS
    big, L = 1 << 36, lib()
    f, b = L.qlora_gated_linear_fwd, L.qlora_gated_linear_bwd
    w = ctypes.byref(_w())

    def fwd(X=FAKE, M=16, w=w, A=FAKE, B=FAKE, r=8, act=0, drop=None, H=FAKE, GU=None, ws=FAKE, n=big):
        return f(X, M, w, A, B, r, 1.0, act, drop, H, GU, ws, n, None)

    def bwd(dH=FAKE, X=FAKE, GU=FAKE, M=16, w=w, A=FAKE, B=FAKE, r=8, act=0, drop=None, dX=FAKE, gd=0, dA=FAKE,
            dB=FAKE, ws=FAKE, n=big):
        return b(dH, X, GU, M, w, A, B, r, 1.0, act, drop, dX, gd, dA, dB, ws, n, None)

    for act in (-1, 2):
        assert fwd(act=act) == BAD and bwd(act=act) == BAD
    for p in BAD_DROPOUT:
        assert fwd(drop=_cfg(p)) == BAD and bwd(drop=_cfg(p)) == BAD
    assert fwd(w=ctypes.byref(_w(768, 256))) == UNS and fwd(w=ctypes.byref(_w(512, 100))) == UNS
    assert fwd(w=ctypes.byref(_w(blocksize=32))) == UNS and fwd(r=136) == UNS and fwd(r=4) == UNS
    assert fwd(X=None) == BAD and fwd(H=None) == BAD and fwd(GU=FAKE + 2) == BAD and fwd(A=None) == BAD
    assert fwd(n=1024) == BAD and fwd(M=-1) == BAD and fwd(M=0, X=None, H=None) == 0
    assert bwd(GU=None) == BAD and bwd(dH=FAKE + 8) == BAD and bwd(gd=7) == BAD and bwd(dA=FAKE + 8) == BAD
    assert bwd(n=1024) == BAD and bwd(w=ctypes.byref(_w(768, 256))) == UNS
    assert bwd(dX=None, r=0, A=None, B=None, dA=None, dB=None) == 0  # nothing asked for


def test_workspace_queries(Q):
    from bit_nf4_quantized_08_b200._lib import lib
    L = lib()
    w = ctypes.byref(_w(1024, 512))
    for M in (1, 64, 65, 2000):
        for bwd in (0, 1):
            assert L.qlora_fused_linear_dropout_workspace(M, w, 2, 16, bwd) >= \
                L.qlora_fused_linear_workspace(M, w, 2, 16, bwd) > 0
            assert L.qlora_gated_linear_workspace(M, w, 16, bwd) > 0
        # the backward holds the gradient of the pre-activations too
        assert L.qlora_gated_linear_workspace(M, w, 16, 1) >= L.qlora_fused_linear_workspace(M, w, 2, 16, 1) + 2 * M * 1024
    assert L.qlora_gated_linear_workspace(5, ctypes.byref(_w(768, 512)), 16, 0) == 0
    assert L.qlora_fused_linear_dropout_workspace(5, w, 2, 12, 0) == 0


def test_python_argument_checks(Q):
    """CPU tensors and malformed shapes are refused before the library is called."""
    w = Q.NF4Weight.empty(512, 256, True, device="cpu")
    X = torch.zeros(4, 256, dtype=torch.bfloat16)
    A, B = torch.zeros(16, 256, dtype=torch.bfloat16), torch.zeros(512, 8, dtype=torch.bfloat16)
    d = Q.Dropout(0.1, 1)
    with pytest.raises(ValueError):
        Q.qlora_dropout(X, d)
    with pytest.raises(TypeError):
        Q.qlora_dropout(X.half(), d)
    with pytest.raises(ValueError):
        Q.qlora_fused_linear_dropout_fwd(X, w, 2, A, B, 1.0, d)
    with pytest.raises(ValueError):
        Q.qlora_gated_linear_fwd(X, w, A, B, 1.0)
    for bad in (Q.Dropout(0.1, -1), Q.Dropout(0.1, 1 << 64), Q.Dropout(0.1, 1, -2),
                Q.Dropout(0.1, 1, 0, torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            bad.c_struct()
