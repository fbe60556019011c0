"""The linear with adapter dropout at few tokens: the same weight as the backward's, for every token count."""
import pytest
import torch

from test_gpu_dropout import _setup

pytestmark = pytest.mark.gpu

FORMATS = [dict(), dict(dq=False), dict(blocksize=128, code_type="fp4", dq_type="e4m3")]


@pytest.mark.parametrize("fmt", FORMATS, ids=["nf4", "no_dq", "fp4_128_e4m3"])
@pytest.mark.parametrize("nseg", [1, 2])
@pytest.mark.parametrize("M", [1, 5, 16, 17, 64])
def test_weight_operand_is_the_dequantized_weight(Q, cuda, M, nseg, fmt):
    """Tokens that are unit vectors read the weight back; with B = 0 the adapter adds nothing: Y is W' bit for bit."""
    S, K, r = 256, 320, 16
    q, inp, _ = _setup(Q, M, nseg, S, K, r, seed=90, **fmt)
    W = Q.qlora_nf4_dequantize(q)
    A, B = inp["A"].cuda(), torch.zeros(nseg * S, r, dtype=torch.bfloat16, device=cuda)
    for k0 in (0, 63, 256, K - 8):
        cols = [(k0 + i) % K for i in range(M)]
        X = torch.zeros(M, K, dtype=torch.bfloat16, device=cuda)
        X[torch.arange(M), cols] = 1.0
        Y = Q.qlora_fused_linear_dropout_fwd(X, q, nseg, A, B, 2.0, Q.Dropout(0.25, 9, k0))
        assert torch.equal(Y, W[:, cols].T.contiguous()), k0
    torch.cuda.synchronize()
    assert Q.qlora_get_last_error() == 0


@pytest.mark.parametrize("M", [1, 3, 16])
def test_one_rounding_of_the_definition(Q, O, cuda, M):
    """Y against fp64 with U rounded to bf16 as the layer's is: its own rounding, 2^-7 / sqrt(12) = 2.26e-3 of the norm
    if every value sat at the bottom of its binade, and fp32 sums of K = 1088 products, below 1e-4; with the rounding
    of U's few values at another border for 1 in 100 of them: 2.4e-3."""
    nseg, S, K, r, s = 2, 1024, 1088, 16, 2.0
    q, inp, _ = _setup(Q, M, nseg, S, K, r, seed=91)
    X, A, B = (inp[k].cuda() for k in ("X", "A", "B"))
    drop = Q.Dropout(0.2, 5, 5)
    Y = Q.qlora_fused_linear_dropout_fwd(X, q, nseg, A, B, s, drop)
    mask = torch.from_numpy(O.dropout_keep(M * K, 0.2, 5, 5).reshape(M, K)).cuda().double()
    U = (s * O.dropout_factor(0.2) * (X.double() * mask) @ A.double().T).bfloat16().double()
    ref = X.double() @ Q.qlora_nf4_dequantize(q).double().T
    for i in range(nseg):
        ref[:, i * S:(i + 1) * S] += U[:, i * r:(i + 1) * r] @ B[i * S:(i + 1) * S].double().T
    torch.cuda.synchronize()
    assert Q.qlora_get_last_error() == 0
    assert float((Y.double() - ref).norm() / ref.norm()) <= 2.4e-3


def test_captured_calls_share_a_workspace(Q, cuda):
    """Two captured calls of few tokens and eager ones of other sizes in one workspace: the bits of calls alone."""
    sets = []
    for i, M in enumerate((3, 16)):
        q, inp, _ = _setup(Q, M, 2, 512, 576, 16, seed=92 + i)
        sets.append((q, *(inp[k].cuda() for k in ("X", "A", "B")), Q.Dropout(0.3, i, 2)))
    n = max(Q.qlora_fused_linear_dropout_workspace(64, s[0], 2, 16, False) for s in sets)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=cuda)

    def call(q, X, A, B, d, w=None):
        return Q.qlora_fused_linear_dropout_fwd(X, q, 2, A, B, 2.0, d, ws=w)

    ref = [call(*s).clone() for s in sets]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(stream):
        for s in sets:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                outs.append(call(*s, ws))
            graphs.append(g)
        for i in (0, 1, 1, 0, 0, 1):
            outs[i].fill_(0)
            graphs[i].replay()
            q, X, A, B, d = sets[1 - i]
            call(q, X.repeat(4, 1), A, B, d, ws)
            stream.synchronize()
            assert torch.equal(outs[i].view(torch.int16), ref[i].view(torch.int16)), i
    assert Q.qlora_get_last_error() == 0
