"""The gated block's gradients in fp16 among other calls: their magnitudes are in memory that every call
of a handle expects to find zero and leaves zero."""
import pytest
import torch

from tests.test_gpu_gated import _formulas
from tests.test_gpu_gated_range import _normal

pytestmark = pytest.mark.gpu

# (rows, columns, K, dH's deviation): with and without scales, tiles cut and not, up to eight rows
CALLS = [(140, 333, 136, 1.0), (300, 520, 264, 300.0), (8, 5000, 512, 2.0 ** -12), (70, 4096, 512, 300.0),
         (1025, 700, 72, 2.0 ** -12), (9, 129, 72, 1.0)]


def _steps(seed):
    gen = torch.Generator().manual_seed(seed)
    steps = []
    for M, N, K, std in CALLS:
        X, Wg, Wu = _normal(gen, M, K, std=2.0 ** -6), _normal(gen, N, K, std=2.0 ** -7), _normal(gen, N, K, std=2.0 ** -7)
        steps.append((X, Wg, Wu, _normal(gen, M, N), _normal(gen, M, N, std=std), _normal(gen, M, N, std=std)))
    return steps


def _fresh(steps):
    return [[torch.full_like(t, float("nan")) for t in s[:3]] for s in steps]


def _run(g, steps, outs, stream=None):
    for s, o in zip(steps, outs):
        g.run_gated_grad(*s, *o, stream=stream)


def _each_alone(steps):
    """Every call through a handle of its own."""
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    outs = _fresh(steps)
    for s, o in zip(steps, outs):
        with Gemm() as g:
            g.run_gated_grad(*s, *o)
            torch.cuda.synchronize()
    return outs


def _same(a, b):
    return all(torch.equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))


def test_calls_of_many_sizes_through_one_handle():
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    steps = _steps(1)
    want = _each_alone(steps)
    for s, o in zip(steps, want):
        # (a few of the gradients themselves pass fp16's largest: infinite are those and no others)
        for t, w in zip(o, _formulas(*s, "silu")[2]):
            assert torch.equal(t.isinf(), w.abs() >= 65520) or (w[t.isinf() != (w.abs() >= 65520)].abs() / 65520 - 1).abs().max() < 2.0 ** -9
            assert not t.isnan().any()
    with Gemm() as g:
        for order in (1, -1, 1):
            outs = _fresh(steps)
            _run(g, steps[::order], outs[::order])
            torch.cuda.synchronize()
            assert _same(outs, want)
        # only some of the gradients in between
        some = _fresh(steps)
        for i, (s, o) in enumerate(zip(steps, some)):
            g.run_gated_grad(*s, dX=o[0]) if i % 2 else g.run_gated_grad(*s, dWg=o[1], dWu=o[2])
        outs = _fresh(steps)
        _run(g, steps, outs)
        assert _same(outs, want)
        assert g.device_status() == (0, 0)


def test_captured_before_the_memory_grows():
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    steps = _steps(2)
    want = _each_alone(steps)
    with Gemm() as g:
        small, first = steps[5:], _fresh(steps[5:])
        stream = torch.cuda.Stream()
        _run(g, small, first, stream=stream)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            _run(g, small, first)
        for _ in range(2):
            outs = _fresh(steps)
            torch.cuda.synchronize()
            _run(g, steps, outs)
            for t in first[0]:
                t.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert _same(outs, want) and _same(first, want[5:])


def test_two_handles_on_two_streams():
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    steps = _steps(3)
    want = _each_alone(steps)
    with Gemm() as a, Gemm() as b:
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        outs = [[_fresh(steps) for _ in range(4)] for _ in streams]
        torch.cuda.synchronize()
        for i in range(4):
            for g, stream, mine in zip((a, b), streams, outs):
                _run(g, steps, mine[i], stream=stream)
        torch.cuda.synchronize()
        assert all(_same(got, want) for mine in outs for got in mine)
        assert a.device_status() == (0, 0) and b.device_status() == (0, 0)


def test_beside_the_adapters_whose_counters_share_the_memory():
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    gen = torch.Generator().manual_seed(4)
    X, W = _normal(gen, 20, 256), _normal(gen, 320, 256, std=2.0 ** -4)
    down, up = _normal(gen, 5, 8, 256, std=2.0 ** -4), _normal(gen, 5, 320, 8)
    ids = torch.randint(-1, 5, (20,), generator=gen).int().cuda()
    steps = _steps(5)
    want = _each_alone(steps)
    with Gemm() as g:
        Y = torch.empty(20, 320, dtype=torch.float16, device="cuda")
        g.run_adapters(X, W, Y, down, up, ids)
        for _ in range(3):
            outs = _fresh(steps)
            again = torch.full_like(Y, float("nan"))
            for s, o in zip(steps, outs):
                g.run_gated_grad(*s, *o)
                g.run_adapters(X, W, again, down, up, ids)
            assert _same(outs, want) and torch.equal(again, Y)
        assert g.device_status() == (0, 0)


@pytest.mark.parametrize("std", [1.0, 300.0])
def test_after_a_wait_that_ran_out(std):
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    gen = torch.Generator().manual_seed(6)
    M, N, K = 300, 520, 264
    X, Wg, Wu = _normal(gen, M, K, std=2.0 ** -6), _normal(gen, N, K, std=2.0 ** -7), _normal(gen, N, K, std=2.0 ** -7)
    large = (_normal(gen, M, N), _normal(gen, M, N, std=300.0), _normal(gen, M, N, std=300.0))
    then = (_normal(gen, M, N), _normal(gen, M, N, std=std), _normal(gen, M, N, std=std))
    with Gemm() as g:
        want = [torch.empty_like(t) for t in (X, Wg, Wu)]
        g.run_gated_grad(X, Wg, Wu, *then, *want)
        torch.cuda.synchronize()
    with Gemm() as g:
        outs = [torch.empty_like(t) for t in (X, Wg, Wu)]
        g.set_wait_limit(50_000_000)
        g.set_test_stall(True)
        g.run_gated_grad(X, Wg, Wu, *large, *outs)
        assert g.device_status()[0] == 5
        g.set_test_stall(False)
        g.set_wait_limit(2_000_000_000)
        g.run_gated_grad(X, Wg, Wu, *then, *outs)
        assert g.device_status() == (0, 0)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
