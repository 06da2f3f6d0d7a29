"""How much of u = s Down x reaches Up u in gemm_run_adapters: its bits, its range, and what
infinities make of it.

Down x is a sum of integers below 2^24, exact in binary32, and every column of Y is one value
of u times a power of two (Up has one value other than zero per row, W is zero).  So Y shows
u as the second product saw it.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

# 40 rows: the kernels for few rows; 700: tiles.  Ranks of one and two blocks of 64 values.
BOTH = pytest.mark.parametrize("M", [40, 700])
RANKS = pytest.mark.parametrize("R", [8, 16, 24, 64, 72, 128])


@pytest.fixture(scope="module")
def g():
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    h = Gemm()
    yield h
    h.close()


def _single(L, N, R, dt, exponents=(-2, 2)):
    """Up whose row n has one value, a power of two, in column n % R; those values."""
    gen = torch.Generator().manual_seed(R)
    power = 2.0 ** torch.randint(exponents[0], exponents[1] + 1, (L, N), generator=gen)
    up = torch.zeros(L, N, R)
    n = torch.arange(N)
    up[:, n, n % R] = power
    return up.to(dt), power


def _case(M, R, dt, out, K=256, N=300, L=5, big=127):
    gen = torch.Generator().manual_seed(M + R)
    X = torch.randint(-big, big + 1, (M, K), generator=gen).to(dt)
    down = torch.randint(-big, big + 1, (L, R, K), generator=gen).to(dt)
    ids = torch.randint(-1, L, (M,), generator=gen, dtype=torch.int32)
    up, power = _single(L, N, R, dt)
    return X, down, up, power, ids


def _u(X, down, ids):
    u = torch.zeros(X.shape[0], down.shape[1], dtype=torch.float64)
    for a in range(len(down)):
        u[ids == a] = X[ids == a].double() @ down[a].double().T
    return u


def _run(g, X, down, up, ids, out, scale=None, N=None):
    N = up.shape[1]
    W = torch.zeros(N, X.shape[1], dtype=X.dtype, device="cuda")
    Y = torch.full((X.shape[0], N), float("nan"), dtype=out, device="cuda")
    g.run_adapters(X.cuda(), W, Y, down.cuda(), up.cuda(), ids.cuda(),
                   scale=None if scale is None else scale.cuda())
    torch.cuda.synchronize()
    assert g.device_status()[0] == 0
    return Y.cpu()


def _columns(u, power, ids, N):
    """u times Up, exactly."""
    R = u.shape[1]
    p = torch.where(ids[:, None] >= 0, power[ids.clamp(min=0).long()], torch.zeros(()))
    return u[:, torch.arange(N) % R] * p.double()


@BOTH
@RANKS
def test_binary32_results_have_every_bit_of_u_with_bf16_inputs(g, M, R):
    X, down, up, power, ids = _case(M, R, torch.bfloat16, torch.float32)
    scale = torch.tensor([1.0, -0.5, 2.0, 1.0, 2.0 ** -40])
    u = _u(X, down, ids)
    assert u.abs().max() < 2 ** 24 and (u % 2 == 1).any()
    u = u * torch.where(ids >= 0, scale[ids.clamp(min=0).long()], torch.ones(())).double()[:, None]
    got = _run(g, X, down, up, ids, torch.float32, scale=scale)
    assert torch.equal(got.double(), _columns(u, power, ids, up.shape[1]))
