"""Rows and columns of gemm_run_adapters that the tensor cores do not serve (infinities and NaN
in Up, values of u far below their row's largest) in every form that the call takes: rows of Y
aligned or not, in place of the binary32 product or not, tiles whole, in halves and cut along K.
Against the formula in 64 bits; tolerances as in test_gpu_adapters."""
import numpy as np
import pytest
import torch

from tests import parity
from tests.test_gpu_adapters import BF16, CODE, F16, F32, TD, _expect, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    h = Gemm()
    yield h
    h.close()


def _spoil(t, N, seed):
    """Infinities in two adapters, a NaN in a third, and rows of X that give u one value 2^-28 of
    the others; the rows that got one."""
    gen = torch.Generator().manual_seed(seed)
    inf, (L, _, R) = float("inf"), t["up"].shape
    t["up"][0, torch.randint(0, N, (5,), generator=gen), 0] = inf
    t["up"][0, N - 1, R - 1] = -inf
    t["up"][L - 1, torch.randint(0, N, (3,), generator=gen), 1] = -inf
    if L > 2:
        t["up"][1, 0, 2] = float("nan")
    # column 0 of X reaches only u's first value, by 2^-14; in every 37th row nothing else does
    t["X"][:, 0] = 0
    t["down"][:, :, 0] = 0
    t["down"][:, 0] = 0
    t["down"][:, 0, 0] = 2.0 ** -14
    rows = torch.arange(min(3, len(t["X"]) - 1), len(t["X"]), 37)
    t["X"][rows, 0] = 2.0 ** -14
    return rows


def _check(got, t, out):
    want, tau = _expect(t)
    got = got.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        finite = np.isfinite(want)
        same = (got == want) | (np.isnan(got) & np.isnan(want))
        bound = parity.ulp_of(np.where(finite, want, 0.0), out) / 2 + np.where(finite, tau, 0.0)
        ok = same | (finite & (np.abs(got - np.where(finite, want, 0.0)) <= bound * (1 + 1e-9)))
    bad = np.argwhere(~ok)
    assert bad.size == 0, (f"{len(bad)} of {ok.size} off, first {bad[0]}: got {got[tuple(bad[0])]}, "
                           f"want {want[tuple(bad[0])]}")
    return want


def _run(g, t, out_dt, offset=0):
    M, N = len(t["X"]), len(t["W"])
    d = {k: None if v is None else v.cuda() for k, v in t.items()}
    flat = torch.full((M * N + offset,), 7.0, dtype=out_dt, device="cuda")
    Y = flat[offset:].view(M, N)
    g.run_adapters(d["X"], d["W"], Y, d["down"], d["up"], d["ids"], scale=d["scale"])
    torch.cuda.synchronize()
    assert g.device_status()[0] == 0
    return Y


def _case(M, N, K, R, L, din, ids, seed):
    t = _inputs(M, N, K, R, L, TD[din], ids, seed=seed)
    rows = _spoil(t, N, seed)
    return t, rows


@pytest.mark.parametrize("M,N,K,R,L,din,dout,ids", [
    # few rows: vectors of Y aligned, not, and in place of the binary32 product; every rank class
    (40, 320, 256, 16, 5, BF16, BF16, "mixed"),
    (40, 321, 256, 24, 5, F16, F16, "mixed"),
    (200, 1000, 520, 32, 7, F16, F32, "mixed"),
    (200, 1001, 520, 64, 7, F16, F32, "runs"),
    (300, 264, 264, 128, 9, F16, BF16, "mixed"),
    (300, 4096, 264, 72, 9, BF16, F32, "mixed"),
    (1, 1024, 2048, 16, 1, F16, F16, "one"),
    (1500, 1001, 136, 8, 70, F16, F16, "mixed"),
    # tiles: whole, half tiles in the last wave, cut along K, rows of Y at any alignment
    (700, 320, 256, 16, 5, F16, F16, "runs"),
    (2560, 2304, 136, 72, 11, F16, F16, "runs"),
    (2560, 2304, 136, 16, 4, F16, F32, "mixed"),
    (600, 300, 8200, 16, 20, F16, BF16, "mixed"),
    (520, 200, 12288, 32, 3, F16, F32, "runs"),
    (2600, 2653, 200, 16, 17, F16, F16, "runs"),
    (1030, 201, 1096, 64, 7, F16, F16, "runs"),
    (2100, 513, 1032, 128, 6, BF16, BF16, "mixed"),
    (4100, 136, 64, 128, 2, BF16, F32, "runs"),
])
def test_every_form_gives_the_formulas_values(g, M, N, K, R, L, din, dout, ids):
    t, rows = _case(M, N, K, R, L, din, ids, seed=M + N + R)
    want = _check(_run(g, t, TD[dout]), t, dout)
    if M > 1:
        assert np.isinf(want).any() and np.isfinite(want).any()


@pytest.mark.parametrize("M", [100, 700])
@pytest.mark.parametrize("dout", [F16, F32])
@pytest.mark.parametrize("offset", [1, 2, 5])
def test_rows_of_y_that_begin_anywhere(g, M, dout, offset):
    t, _ = _case(M, 264, 512, 16, 6, F16, "mixed", seed=M + offset)
    _check(_run(g, t, TD[dout], offset), t, dout)


def test_forced_configurations(g):
    few, many = (_case(M, 520, 1024, 16, 6, F16, "mixed", seed=M)[0] for M in (100, 700))
    try:
        for t, cfgs in ((few, (dict(variant=1), dict(splits=3), dict(variant=2, max_ctas=10))),
                        (many, (dict(splits=3), dict(splits=-1), dict(group_m=1), dict(max_ctas=6),
                                dict(chain_kblocks=3)))):
            for cfg in cfgs:
                g.set_config(**cfg)
                for out in (F16, F32):
                    _check(_run(g, t, TD[out]), t, out)
    finally:
        g.reset_config()


@pytest.mark.parametrize("M", [300, 900])
@pytest.mark.parametrize("dout", [F16, BF16, F32])
def test_results_repeat(g, M, dout):
    t, _ = _case(M, 1000, 520, 32, 12, F16, "mixed", seed=M)
    first = _run(g, t, TD[dout])
    for _ in range(5):
        again = _run(g, t, TD[dout])
        assert torch.equal(first.view(torch.uint8), again.view(torch.uint8))


@pytest.mark.parametrize("M,N,K,R,L,din,dout,ids", [
    (40, 320, 256, 16, 5, F16, F16, "mixed"),
    (200, 1001, 520, 64, 7, F16, F32, "runs"),
    (300, 264, 264, 128, 9, F16, BF16, "mixed"),
    (1500, 1001, 136, 8, 70, F16, F32, "mixed"),
    (700, 320, 256, 16, 5, F16, F16, "runs"),
    (2560, 2304, 136, 72, 11, F16, F16, "runs"),
    (600, 300, 8200, 16, 20, F16, F32, "mixed"),
    (2600, 2653, 200, 16, 17, F16, F16, "runs"),
])
def test_rows_that_no_window_reaches_beside_rows_that_one_does(g, M, N, K, R, L, din, dout, ids):
    # u's first value is 2^-28 of the others in some rows, 2^-48 in others, in some neither
    t, rows = _case(M, N, K, R, L, din, ids, seed=M + R)
    t["down"][:, 0, 0] = 2.0 ** -24
    t["X"][:, 0] = 0
    t["X"][rows, 0] = 2.0 ** -4
    t["X"][rows[::2], 0] = 2.0 ** -24
    t["X"][::3, 0] = 0
    _check(_run(g, t, TD[dout]), t, dout)


@pytest.mark.parametrize("M,ids", [(100, "mixed"), (2200, "runs")])
@pytest.mark.parametrize("dout", [F16, F32])
def test_an_adapter_with_a_nearly_dead_rank(g, M, ids, dout):
    # every row has a value in the second window, and in each a column of Y that is that value's
    # alone: the dead rank's own bits have to be there
    gen = torch.Generator().manual_seed(M)
    K, N, R, L = 256, 264, 16, 4
    X = torch.randint(-8, 9, (M, K), generator=gen).half()
    down = torch.randint(-8, 9, (L, R, K), generator=gen).half()
    down[:, 5] = (torch.randint(-8, 9, (L, K), generator=gen) * 2.0 ** -20).half()
    up = torch.zeros(L, N, R).half()
    up[:, :, 5] = 64.0
    up[:, 100:, 2] = 0.25
    which = torch.randint(0, L, (M,), generator=gen, dtype=torch.int32)
    which = which if ids == "mixed" else torch.sort(which).values
    u = torch.stack([down[a].double() @ x.double() for a, x in zip(which.tolist(), X)])
    want = torch.empty(M, N, dtype=torch.float64)
    want[:, :100] = 64 * u[:, 5:6]
    want[:, 100:] = 64 * u[:, 5:6] + u[:, 2:3] / 4
    Y = torch.empty(M, N, dtype=torch.float16 if dout == F16 else torch.float32, device="cuda")
    W = torch.zeros(N, K, dtype=torch.float16, device="cuda")
    g.run_adapters(X.cuda(), W, Y, down.cuda(), up.cuda(), which.cuda())
    torch.cuda.synchronize()
    assert g.device_status() == (0, 0)
    # integers (times 2^-20 for the dead rank) that both parts hold exactly
    assert torch.equal(Y.cpu(), want.float().to(Y.dtype).cpu())
