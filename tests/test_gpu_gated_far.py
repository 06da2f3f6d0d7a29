"""The gated block's gradients for gates as far from zero as bf16 holds them.  From |g| = 10^4 on
every activation is g or 0 and its derivative 1 or 0, in 64 bits as well as exactly, and the factors
here are powers of two: results are exact."""
import pytest
import torch

from tests.test_gpu_gated import KINDS, g  # noqa: F401

pytestmark = pytest.mark.gpu

FAR = [1e4, 1e6, 1e10, 1e13, 2e13, 1e14, 1e18, 1e20, 1e30, 2e38, 3e38]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [1, 5, 8, 9, 136])
def test_gates_far_from_zero(g, kind, M):  # noqa: F811
    bf = torch.bfloat16
    gate = torch.tensor([s * v for v in FAR for s in (1.0, -1.0)], device="cuda").to(bf).expand(M, -1).contiguous()
    N = gate.shape[1]
    assert torch.isfinite(gate).all()
    up, dH = torch.full_like(gate, 4.0), torch.full_like(gate, 0.25)
    # row m of X is the m-th unit vector, and none of dU reaches dX
    X = torch.eye(M, 136, device="cuda", dtype=bf)
    Wg, Wu = torch.ones(N, 136, device="cuda", dtype=bf), torch.zeros(N, 136, device="cuda", dtype=bf)
    dX, dWg, dWu = torch.empty_like(X), torch.empty_like(Wg), torch.empty_like(Wu)
    g.run_gated_grad(X, Wg, Wu, gate, up, dH, dX, dWg, dWu, activation=kind)
    slope = (gate[0] > 0).float()
    assert torch.equal(dX, torch.full_like(dX, float(slope.sum())))
    assert torch.equal(dWg[:, :M].float(), slope[:, None].expand(N, M)) and not dWg[:, M:].any()
    want = (gate[0].float() * 0.25 * slope).to(bf)
    assert torch.equal(dWu[:, :M], want[:, None].expand(N, M)) and not dWu[:, M:].any()
    # a NaN stays one, in its own row of dX and of the weights' gradients
    gate[0, 3] = float("nan")
    if kind != "relu":
        g.run_gated_grad(X, Wg, Wu, gate, up, dH, dX, dWg, dWu, activation=kind)
        assert dX[0].isnan().all() and dX[1:].isfinite().all()
        rest = torch.arange(N, device="cuda") != 3
        assert dWg[3].isnan().any() and dWg[rest].isfinite().all() and dWu[rest].isfinite().all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [3, 200])
def test_projections_far_from_zero(g, kind, M):  # noqa: F811
    """H of such projections: act(G) U with G = 2^(60 + e) and its negative, U = 2^-50."""
    bf = torch.bfloat16
    e = torch.tensor([14.0, 20.0, 40.0, 60.0, 62.0])
    X = torch.zeros(M, 8, device="cuda", dtype=bf)
    X[:, 0] = 2.0 ** 60
    N = 2 * len(e)
    Wg, Wu = torch.zeros(N, 8, device="cuda", dtype=bf), torch.zeros(N, 8, device="cuda", dtype=bf)
    Wg[:, 0] = torch.cat([2.0 ** e, -(2.0 ** e)]).to(bf).cuda()
    Wu[:, 0] = 2.0 ** -110
    H = torch.empty(M, N, device="cuda", dtype=bf)
    g.run_gated(X, Wg, Wu, H, activation=kind)
    want = torch.cat([2.0 ** (10 + e), torch.zeros(len(e))]).cuda()
    assert torch.equal(H.float(), want.expand(M, N))
