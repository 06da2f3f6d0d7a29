"""A handle's own device memory under the operators and the product: first calls on any
stream, and graphs that outlive its growth."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _adapted(M, N=520, K=1024, R=16, L=20):
    """Inputs of integers so small that binary32 sums of them are exact, and the result."""
    gen = torch.Generator().manual_seed(M)

    def ints(*shape):
        return torch.randint(-2, 3, shape, generator=gen).bfloat16().cuda()
    X, W, down, up = ints(M, K), ints(N, K), ints(L, R, K), ints(L, N, R)
    ids = torch.randint(-1, L, (M,), generator=gen, dtype=torch.int32).cuda()
    want = X.double() @ W.double().T
    for a in range(L):
        r = ids == a
        u = X[r].double() @ down[a].double().T
        assert u.abs().max() < 2 ** 16 if r.any() else True
        want[r] += u @ up[a].double().T
    return X, W, down, up, ids, want


def _near(Y, want):
    # u's 16 bits carry these integers only in part: 2^-16 of at most 16 terms of 2 |u|, and
    # a rounding of the result
    return (Y.double() - want).abs().max() <= 2.0 ** -16 * 16 * 2 * 2 ** 10 + 2.0 ** -23 * want.abs().max()


@pytest.mark.parametrize("M", [40, 600])
def test_first_call_on_a_side_stream_while_the_default_one_is_busy(M):
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    X, W, down, up, ids, want = _adapted(M, K=8192 if M == 600 else 1024)
    Y = torch.full(want.shape, float("nan"), device="cuda")
    big = torch.randn(8192, 8192, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with Gemm() as g:
            for _ in range(20):
                big @ big                      # some 12 ms of the default stream
            g.run_adapters(X, W, Y, down, up, ids, stream=side)
            side.synchronize()
            got = Y.clone()
            assert g.device_status(stream=side) == (0, 0)
            torch.cuda.synchronize()
            assert _near(got, want)
            Y.fill_(float("nan"))
            torch.cuda.synchronize()
            g.run_adapters(X, W, Y, down, up, ids, stream=side)
            side.synchronize()
            assert _near(Y, want)


def test_a_captured_graph_replays_after_larger_calls_of_its_handle():
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    small, large = _adapted(64), _adapted(8192, N=1040)
    Y, Z = (torch.empty(t[5].shape, device="cuda") for t in (small, large))
    A, B = small[0].new_ones(256, 16384), small[0].new_ones(200, 16384)
    C, D = torch.empty(256, 200, device="cuda"), torch.empty(1024, 1000, device="cuda")
    with Gemm() as g:
        def step():
            g.run_adapters(*small[:2], Y, *small[2:5])
            g.run(A, B, C)                     # cut along K: workspace and counters
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        g.run_adapters(*large[:2], Z, *large[2:5])
        g.run(A.new_ones(1024, 16384), A.new_ones(1000, 16384), D)
        other = torch.full((1 << 26,), float("nan"), device="cuda")   # what freed memory would hold
        torch.cuda.synchronize()
        for _ in range(3):
            Y.fill_(float("nan"))
            C.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert _near(Y, small[5]) and (C == 16384).all()
        assert _near(Z, large[5]) and (D == 16384).all()
        assert torch.isnan(other).all()
        assert g.device_status() == (0, 0)
