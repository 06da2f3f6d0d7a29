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


def _powers(M, R, L, dt, low, high, gen):
    """X, Down and ids whose u[i][r] is one product of two values of their type, of a size
    between 2^low and 2^high (both reached in most rows), by one value other than zero in
    every row of Down."""
    K = 8 * ((R + 7) // 8)
    ids = torch.randint(0, L, (M,), generator=gen, dtype=torch.int32)
    half = torch.randint(low // 2, high // 2 + 1, (L, R), generator=gen)
    half[:, 0], half[:, 1] = high // 2, low // 2
    at = torch.stack([torch.randperm(K, generator=gen)[:R] for _ in range(L)])
    down = torch.zeros(L, R, K)
    down.scatter_(2, at[:, :, None], ((1 + torch.rand(L, R, generator=gen)) * 2.0 ** half)[:, :, None])
    X = torch.zeros(M, K)
    X.scatter_(1, at[ids.long()], 2.0 ** half[ids.long()] * (1 + torch.rand(M, R, generator=gen))
               * (1 - 2 * torch.randint(0, 2, (M, R), generator=gen)))
    return X.to(dt), down.to(dt), ids


def _each_value(g, X, down, ids, R, out, relative):
    """Every column of Y is u's value times a power of two to within `relative` of it, and a
    rounding."""
    N = 300
    up, power = _single(len(down), N, R, X.dtype)
    u = _u(X, down, ids)
    want = _columns(u, power, ids, N)
    got = _run(g, X, down, up, ids, out).double()
    ulp = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[out]
    # rows whose u binary32 holds, and what it holds of their results (past its end: infinity)
    end = 2.0 ** 128 * (1 - 2.0 ** -25)
    rows = (u.abs() < end).all(dim=1)
    got, want = got[rows], want[rows]
    over = want.abs() >= end
    assert rows.any() and (got[over] == want[over].sign() * float("inf")).all()
    got, want = got[~over], want[~over]
    assert ((got - want).abs() <= (relative + ulp * (1 + relative)) * want.abs()).all()
    return u


@BOTH
@RANKS
@pytest.mark.parametrize("out,relative", [(torch.float32, 2.0 ** -20), (torch.bfloat16, 2.0 ** -17)])
@pytest.mark.parametrize("low,high", [(-24, 20), (-8, 18), (-28, -10), (4, 22)])
def test_values_far_below_their_rows_largest_survive_in_fp16(g, M, R, out, relative, low, high):
    X, down, ids = _powers(M, R, 5, torch.float16, low, high, torch.Generator().manual_seed(R + M + high))
    u = _each_value(g, X, down, ids, R, out, relative)
    assert u.abs().max() / u[u != 0].abs().min() > 2.0 ** (high - low - 2)


@BOTH
@RANKS
@pytest.mark.parametrize("low,high", [(-124, -80), (-120, 60), (-60, 120), (90, 126)])
def test_binary32_results_have_every_value_of_u_with_bf16_inputs(g, M, R, low, high):
    X, down, ids = _powers(M, R, 5, torch.bfloat16, low, high, torch.Generator().manual_seed(R + M + high))
    _each_value(g, X, down, ids, R, torch.float32, 0.0)


@BOTH
def test_large_values_in_up_with_bf16_inputs(g, M):
    # Up of 2^126 times u of 2^-30: eight such terms are far from binary32's end
    K, N, R, L = 64, 130, 8, 2
    X = torch.zeros(M, K).bfloat16()
    X[:, 0] = 2.0 ** -15
    down = torch.zeros(L, R, K).bfloat16()
    down[:, :, 0] = 2.0 ** -15
    up = torch.full((L, N, R), 2.0 ** 126).bfloat16()
    ids = torch.zeros(M, dtype=torch.int32)
    for out in (torch.float32, torch.bfloat16):
        assert (_run(g, X, down, up, ids, out) == 8 * 2.0 ** 96).all()


def test_a_row_with_one_wide_value_leaves_the_other_rows_bits(g):
    # (the row is multiplied in binary32, its neighbours in the tensor cores as before)
    for M in (40, 700):
        gen = torch.Generator().manual_seed(M)
        X = torch.randn(M, 256, generator=gen).half()
        down = (torch.randn(3, 16, 256, generator=gen) / 16).half()
        up = torch.randn(3, 200, 16, generator=gen).half()
        ids = torch.randint(0, 3, (M,), generator=gen, dtype=torch.int32)
        before = _run(g, X, down, up, ids, torch.float32)
        X[7] = 0
        X[7, 0] = 2.0 ** -24
        down[:, :, 0], down[:, 0, 0] = 2.0 ** -10, 2.0 ** 15
        X2 = X.clone()
        X2[:, 0] = 0
        X2[7, 0] = X[7, 0]
        rows = torch.arange(M) != 7
        a = _run(g, X2, down, up, ids, torch.float32)
        X2[7, 0] = 0
        b = _run(g, X2, down, up, ids, torch.float32)
        assert torch.equal(a[rows], b[rows]) and (b[7] == 0).all()
        u = _u(X, down, ids)[7]
        want = (up[ids[7].item()].double() * u).sum(-1)
        mag = (up[ids[7].item()].double() * u).abs().sum(-1)
        assert ((a[7].double() - want).abs() <= 17 * 2.0 ** -24 * mag).all()
        assert torch.isfinite(before).all()


def test_an_infinity_at_the_start_of_one_adapter_leaves_the_end_of_the_one_before(g):
    # (in the tiles, columns past N meet the next adapter's rows of Up)
    gen = torch.Generator().manual_seed(17)
    for M in (40, 900):
        X = torch.randn(M, 256, generator=gen).bfloat16()
        down = (torch.randn(4, 16, 256, generator=gen) / 16).bfloat16()
        up = torch.randn(4, 300, 16, generator=gen).bfloat16()
        ids = torch.randint(0, 4, (M,), generator=gen, dtype=torch.int32)
        for out in (torch.bfloat16, torch.float32):
            before = _run(g, X, down, up, ids, out)
            spoilt = up.clone()
            spoilt[1:, :6] = float("inf")
            got = _run(g, X, down, spoilt, ids, out)
            assert torch.equal(got[ids == 0], before[ids == 0])
            assert torch.equal(got[:, 32:], before[:, 32:])
