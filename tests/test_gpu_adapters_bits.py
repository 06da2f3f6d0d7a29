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


@BOTH
@pytest.mark.parametrize("R", [8, 24, 64, 128])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out", ["same", torch.float32])
def test_infinities_in_up_give_what_the_formula_gives(g, M, R, dt, out):
    # small integers, so that every finite sum is exact and each result is the formula's
    # value rounded once; u is often zero, often exact in one part and of either sign
    out = dt if out == "same" else out
    gen = torch.Generator().manual_seed(M + 3 * R)
    K, N, L = 64, 300, 6
    X = torch.randint(-3, 4, (M, K), generator=gen).to(dt)
    X[::7, 8:] = 0
    down = torch.randint(-2, 3, (L, R, K), generator=gen).to(dt)
    down[:, 1] = torch.randint(-120, 121, (L, K), generator=gen).to(dt)
    up = torch.randint(-2, 3, (L, N, R), generator=gen).to(dt)
    inf = float("inf")
    up[0, 0, 0], up[0, 40, 1], up[0, 299, R - 1] = inf, -inf, inf
    up[1, 7, 0], up[1, 7, 3] = inf, -inf               # of one or of both signs, by u
    up[2, 130, :] = inf
    up[3, 64:70, 2] = -inf
    up[3, 65, 5] = float("nan")
    ids = torch.randint(-1, L, (M,), generator=gen, dtype=torch.int32)
    W = torch.randint(-2, 3, (N, K), generator=gen).to(dt)
    u = _u(X, down, ids)
    assert u.abs().max() < 2 ** 16 and (u == 0).any()
    want = X.double() @ W.double().T
    for a in range(L):
        r = ids == a
        want[r] += (u[r][:, None, :] * up[a].double()).sum(-1)
    finite = want[torch.isfinite(want)]
    assert finite.abs().max() < 2 ** 24 and want.isinf().any() and want.isnan().any()
    Y = torch.full((M, N), 7.0, dtype=out, device="cuda")
    g.run_adapters(X.cuda(), W.cuda(), Y, down.cuda(), up.cuda(), ids.cuda())
    torch.cuda.synchronize()
    got, want = Y.cpu(), want.float().to(out)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(nan=0.0, posinf=inf, neginf=-inf),
                       want.nan_to_num(nan=0.0, posinf=inf, neginf=-inf))


@BOTH
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_infinities_and_nan_in_x_give_what_the_formula_gives(g, M, dt):
    # u of row 5 has infinities, row 9's has NaN; two values of the others are infinite
    gen = torch.Generator().manual_seed(M)
    K, N, R, L = 64, 130, 16, 3
    X = torch.randint(-3, 4, (M, K), generator=gen).to(dt)
    down = torch.randint(-2, 3, (L, R, K), generator=gen).to(dt)
    down[:, :, 5] = 0
    down[:, 2, 5], down[:, 3, 5] = 1, -1
    up = torch.randint(-2, 3, (L, N, R), generator=gen).to(dt)
    up[:, :, 2] = torch.randint(1, 3, (L, N), generator=gen).to(dt)
    up[:, :60, 3] = 0                                   # infinity times zero: NaN
    up[:, 60:, 3] = -1
    up[1, 100, 4] = float("inf")
    ids = torch.randint(0, L, (M,), generator=gen, dtype=torch.int32)
    ids[5], ids[9] = 1, 2
    X[5, 5], X[9, 5] = float("inf"), float("nan")
    u = torch.stack([(down[int(a)].double() * x.double()).sum(-1) for a, x in zip(ids, X)])
    # (infinity times the zeros of Down: NaN in every other value of u, as the formula has it)
    want = torch.stack([(up[int(a)].double() * v).sum(-1) for a, v in zip(ids, u)])
    Y = torch.full((M, N), 7.0, dtype=torch.float32, device="cuda")
    g.run_adapters(X.cuda(), torch.zeros(N, K, dtype=dt, device="cuda"), Y, down.cuda(), up.cuda(),
                   ids.cuda())
    torch.cuda.synchronize()
    got = Y.cpu()
    rows = torch.ones(M, dtype=torch.bool)
    rows[[5, 9]] = False
    assert torch.isnan(got[[5, 9]]).all() and torch.isnan(want[[5, 9]]).all()
    same = got[rows].double() == want[rows]
    both = torch.isnan(got[rows]) & torch.isnan(want[rows])
    assert (same | both).all()
