"""The gated block's gradients where dG = dH U act'(G) and dU = dH act(G) leave fp16's range, or lie
below its normal numbers, and the gradients do not.

Tolerances, for each element of a result: every term is off by half a step of itself (`half`, and
2^-17 for its evaluation, as in test_gpu_gated) or, where that is more, by 2^-21 of the largest
|dG| and |dU| of its row of dX, or of its column for the weights' gradients, times its factor; the
result is rounded once.  Up to eight rows' weights' gradients have no such term."""
import pytest
import torch

from tests import parity
from tests.test_gpu_gated import _formulas, g  # noqa: F401

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -11
FLOOR = 2.0 ** -21


def _normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen) * std).half().cuda()


def _new(X, W):
    return [torch.full_like(t, float("nan")) for t in (X, W, W)]


def _check(X, Wg, Wu, gate, up, dH, outs, kind):
    dG, dU, want = _formulas(X, Wg, Wu, gate, up, dH, kind)
    few = X.shape[0] <= 8
    row = torch.maximum(dG.abs(), dU.abs()).amax(1, keepdim=True)
    ag, au, x = Wg.double().abs(), Wu.double().abs(), X.double().abs()
    bounds = [(HALF + 2.0 ** -17) * (dG.abs() @ ag + dU.abs() @ au) + FLOOR * row * (ag + au).sum(0)]
    for d in (dG, dU):
        column = 0.0 if few else FLOOR * d.abs().amax(0)[:, None]
        bounds.append((HALF + 2.0 ** -17) * (d.abs().T @ x) + column * x.sum(0))
    for name, got, w, b in zip(("dX", "dWg", "dWu"), outs, want, bounds):
        assert w.abs().max() < 60000, "the gradients themselves have to be in range"
        w, b = w.cpu(), b.cpu()
        step = torch.from_numpy(parity.ulp_of((w.abs() + b).numpy(), 0))
        off = (got.double().cpu() - w).abs()
        bad = (~(off <= (step / 2 + b) * (1 + 1e-9))).nonzero()
        assert len(bad) == 0, (name, len(bad), bad[0].tolist(), float(got[tuple(bad[0])]), float(w[tuple(bad[0])]),
                               float(b[tuple(bad[0])]))


def _run(g, X, Wg, Wu, gate, up, dH, kind):  # noqa: F811
    outs = _new(X, Wg)
    g.run_gated_grad(X, Wg, Wu, gate, up, dH, *outs, activation=kind)
    # whichever others are asked for, and once more
    some = _new(X, Wg)
    g.run_gated_grad(X, Wg, Wu, gate, up, dH, dX=some[0], activation=kind)
    g.run_gated_grad(X, Wg, Wu, gate, up, dH, dWg=some[1], dWu=some[2], activation=kind)
    again = _new(X, Wg)
    g.run_gated_grad(X, Wg, Wu, gate, up, dH, *again, activation=kind)
    for a, b, c in zip(outs, some, again):
        assert torch.equal(a, b) and torch.equal(a, c)
    return outs


SIZES = [(1, 200, 72), (8, 1001, 136), (9, 1001, 136), (100, 5001, 1024), (300, 520, 264), (1025, 1401, 136)]


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_slopes_beyond_the_largest_number(g, M, N, K, kind):  # noqa: F811
    # dG up to 10^6 and dU up to 10^5, factors so small that the sums stay in range
    gen = torch.Generator().manual_seed(M + N)
    X, Wg, Wu = _normal(gen, M, K, std=2.0 ** -8), _normal(gen, N, K, std=2.0 ** -9), _normal(gen, N, K, std=2.0 ** -9)
    gate, up, dH = _normal(gen, M, N, std=2.0), _normal(gen, M, N, std=300.0), _normal(gen, M, N, std=300.0)
    _check(X, Wg, Wu, gate, up, dH, _run(g, X, Wg, Wu, gate, up, dH, kind), kind)


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("M,N,K", SIZES + [(4096, 136, 72)])
def test_slopes_below_the_smallest_number(g, M, N, K, kind):  # noqa: F811
    # dG and dU of some 10^-8 and less, of one sign, and factors whose sums are in range
    gen = torch.Generator().manual_seed(M + N)
    X, Wg, Wu = (_normal(gen, r, K).abs() * 30 for r in (M, N, N))
    gate, up = _normal(gen, M, N).abs() * 2.0 ** -4 + 0.05, _normal(gen, M, N).abs() * 2.0 ** -12
    dH = _normal(gen, M, N).abs() * 2.0 ** -13
    outs = _run(g, X, Wg, Wu, gate, up, dH, kind)
    _check(X, Wg, Wu, gate, up, dH, outs, kind)
    assert all((o > 0).any() for o in outs)


@pytest.mark.parametrize("kind", ["silu", "relu"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_rows_and_columns_of_their_own_magnitudes(g, M, N, K, kind):  # noqa: F811
    """Magnitudes of 2^-14 to 2^8 row by row (dH) and of as much column by column (up): what is large
    in one row or column takes nothing from another.  The factors even out what they can."""
    gen = torch.Generator().manual_seed(M + N)
    rows = 2.0 ** (torch.randint(-14, 9, (M, 1), generator=gen).float())
    cols = 2.0 ** (torch.randint(-10, 5, (1, N), generator=gen).float())
    gate = _normal(gen, M, N)
    up = (torch.randn(M, N, generator=gen) * cols).half().cuda()
    dH = (torch.randn(M, N, generator=gen) * rows).half().cuda()
    if M > 3:
        dH[2] = 0.0                                      # a row, and a column, of nothing
        up[:, N // 2], gate[:, N // 2] = 0.0, 0.0
    X = (torch.randn(M, K, generator=gen) / rows * 2.0 ** -4).half().cuda()
    Wg, Wu = (torch.randn(N, K, generator=gen) / cols.T * 2.0 ** -5).half().cuda(), _normal(gen, N, K, std=2.0 ** -5)
    outs = _run(g, X, Wg, Wu, gate, up, dH, kind)
    _check(X, Wg, Wu, gate, up, dH, outs, kind)
    if M > 3:
        assert not outs[0][2].any() and not outs[1][N // 2].any() and not outs[2][N // 2].any()


@pytest.mark.parametrize("M", [5, 300])
def test_what_is_not_finite_stays_where_it_is(g, M):  # noqa: F811
    """An infinity and a NaN among slopes that have to be scaled: its row of dX, its column's rows of the
    weights' gradients, and nothing else."""
    gen = torch.Generator().manual_seed(M)
    N, K = 200, 72
    X, Wg, Wu = _normal(gen, M, K, std=2.0 ** -8), _normal(gen, N, K, std=2.0 ** -9), _normal(gen, N, K, std=2.0 ** -9)
    gate, up, dH = _normal(gen, M, N, std=2.0), _normal(gen, M, N, std=300.0), _normal(gen, M, N, std=300.0)
    clean = _run(g, X, Wg, Wu, gate, up, dH, "silu")
    dH[1, 7], up[3, 100] = float("inf"), float("nan")
    outs = _new(X, Wg)
    g.run_gated_grad(X, Wg, Wu, gate, up, dH, *outs, activation="silu")
    rows, cols = torch.ones(M, dtype=torch.bool), torch.ones(N, dtype=torch.bool)
    rows[[1, 3]], cols[[7, 100]] = False, False
    assert torch.equal(outs[0][rows], clean[0][rows]) and not outs[0][~rows].isfinite().any()
    assert torch.equal(outs[1][cols], clean[1][cols]) and not outs[1][~cols].isfinite().any()
    cols[100] = True                                     # (up is no factor of dU)
    assert torch.equal(outs[2][cols], clean[2][cols]) and not outs[2][7].isfinite().any()


def test_replayed_with_slopes_of_another_range(g):  # noqa: F811
    # one captured call, inputs from ordinary to far and back
    gen = torch.Generator().manual_seed(4)
    M, N, K = 140, 333, 136
    X, Wg, Wu = _normal(gen, M, K, std=2.0 ** -6), _normal(gen, N, K, std=2.0 ** -7), _normal(gen, N, K, std=2.0 ** -7)
    gate, up, dH = _normal(gen, M, N), _normal(gen, M, N), _normal(gen, M, N)
    outs = _new(X, Wg)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        g.run_gated_grad(X, Wg, Wu, gate, up, dH, *outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        g.run_gated_grad(X, Wg, Wu, gate, up, dH, *outs)
    for std in (1.0, 300.0, 2.0 ** -12, 1.0, 2.0 ** -12, 300.0):
        up.copy_(_normal(gen, M, N, std=std))
        dH.copy_(_normal(gen, M, N, std=std))
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        _check(X, Wg, Wu, gate, up, dH, outs, "silu")
        other = _new(X, Wg)
        g.run_gated_grad(X, Wg, Wu, gate, up, dH, *other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, other))
    assert g.device_status() == (0, 0)
