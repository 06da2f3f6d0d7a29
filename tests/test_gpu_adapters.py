"""Projections with a low-rank adapter per row (gemm_run_adapters) against the formula in
64 bits:  Y[i] = W x_i + s_a Up_a (Down_a x_i),  a = row_adapter[i].

Tolerance.  Both products of length K accumulate in binary32: tau = 8 * 2^-24 * sqrt(K) *
sigma for the shared product (parity.tau_of) and the same, tau_u, for every value of
u = Down x.  The second product carries tau_u through |s Up|, and its own error: u enters it
with at least 17 significant bits (|e| <= 2^-18 |u|) and its at most 128 terms add in
binary32 (<= 2^-17 of the terms' sum), together below 2^-16 * sum |s u up|.  Then one
rounding of the sum, ulp / 2.
"""
import numpy as np
import pytest
import torch

import seeded_inputs as si
from tests import parity

pytestmark = pytest.mark.gpu

F16, BF16, F32 = 0, 1, 2
TD = si.TORCH_DTYPE
CODE = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}


@pytest.fixture(scope="module")
def g():
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    h = Gemm()
    yield h
    h.close()


def _inputs(M, N, K, R, L, dt, ids, seed, scale=True):
    gen = torch.Generator().manual_seed(seed)
    t = dict(X=torch.randn(M, K, generator=gen).to(dt),
             W=(torch.randn(N, K, generator=gen) * K ** -0.5).to(dt),
             down=(torch.randn(L, R, K, generator=gen) * K ** -0.5).to(dt),
             up=(torch.randn(L, N, R, generator=gen) * 0.1).to(dt),
             scale=(torch.rand(L, generator=gen) * 3 - 1) if scale else None)
    if ids == "mixed":
        t["ids"] = torch.randint(-1, L, (M,), generator=gen, dtype=torch.int32)
    elif ids == "none":
        t["ids"] = torch.full((M,), -1, dtype=torch.int32)
    elif ids == "one":
        t["ids"] = torch.full((M,), L - 1, dtype=torch.int32)
    else:  # runs of rows
        cut = torch.sort(torch.randint(0, M + 1, (L,), generator=gen)).values
        t["ids"] = (torch.bucketize(torch.arange(M), cut, right=True) - 1).to(torch.int32)
    return t


def _expect(t):
    """The formula in 64 bits, and the bound on everything before the rounding."""
    X, W = t["X"].double().numpy(), t["W"].double().numpy()
    down, up = t["down"].double().numpy(), t["up"].double().numpy()
    ids, K = t["ids"].numpy(), X.shape[1]
    scale = np.ones(len(down)) if t["scale"] is None else t["scale"].double().numpy()
    base = X @ W.T
    tau = parity.tau_of(np.sqrt((X ** 2) @ (W ** 2).T), K)
    term = np.zeros_like(base)
    for a in set(ids.tolist()):
        if not 0 <= a < len(down):
            continue
        r = ids == a
        u = X[r] @ down[a].T
        tau_u = parity.tau_of(np.sqrt((X[r] ** 2) @ (down[a] ** 2).T), K)
        term[r] = scale[a] * (u @ up[a].T)
        tau[r] += abs(scale[a]) * ((tau_u + 2.0 ** -16 * np.abs(u)) @ np.abs(up[a]).T)
    return base + term, tau


def _check(got, want, tau, out):
    got = got.double().cpu().numpy()
    bound = parity.ulp_of(want, out) / 2 + tau
    err = np.abs(got - want)
    bad = np.argwhere(~(err <= bound * (1 + 1e-9)))
    assert bad.size == 0, (f"{len(bad)} of {err.size} off, first {bad[0]}: got {got[tuple(bad[0])]}, "
                           f"want {want[tuple(bad[0])]} +- {bound[tuple(bad[0])]}")


def _run(g, t, out_dt, **kw):
    d = {k: None if v is None else v.cuda() for k, v in t.items()}
    Y = torch.full((t["X"].shape[0], t["W"].shape[0]), float("nan"), dtype=out_dt, device="cuda")
    g.run_adapters(d["X"], d["W"], Y, d["down"], d["up"], d["ids"], scale=d["scale"], **kw)
    torch.cuda.synchronize()
    return Y


@pytest.mark.parametrize("M,N,K,R,L,din,dout,ids", [
    (1, 256, 512, 16, 3, BF16, BF16, "one"),
    (1, 1, 8, 8, 1, F16, F32, "one"),
    (2, 129, 72, 8, 5, F16, F16, "mixed"),
    (7, 1000, 1000, 24, 2, BF16, F32, "mixed"),
    (33, 320, 4104, 32, 40, F16, BF16, "mixed"),
    (127, 513, 264, 40, 64, BF16, BF16, "mixed"),
    (128, 384, 1024, 16, 128, BF16, BF16, "mixed"),
    (129, 257, 640, 64, 4, F16, F16, "runs"),
    (200, 1001, 2008, 24, 13, F16, F32, "mixed"),
    (256, 640, 8192, 16, 200, BF16, BF16, "mixed"),
    (300, 264, 512, 128, 9, BF16, BF16, "mixed"),
    (300, 129, 192, 120, 3, F16, F32, "runs"),
    (700, 392, 328, 16, 6, BF16, BF16, "runs"),
    (1030, 200, 1096, 64, 7, F16, F16, "runs"),
    (2100, 1032, 264, 32, 5, BF16, BF16, "runs"),
    (2100, 1001, 264, 8, 300, BF16, BF16, "mixed"),
    (2049, 130, 520, 56, 3, F16, F32, "mixed"),
    (64, 512, 512, 16, 4, BF16, BF16, "none"),
    (2500, 512, 512, 16, 4, BF16, BF16, "none"),
    (4100, 136, 64, 128, 2, BF16, BF16, "runs"),
    # the product cut along K, into half tiles in its last wave, of several chains, of one
    # short K block; more adapters in a tile than one group of accumulator columns holds
    (600, 300, 8200, 16, 40, BF16, BF16, "mixed"),
    (2560, 2304, 136, 72, 11, F16, F16, "runs"),
    (513, 1000, 8, 8, 3, BF16, F32, "mixed"),
    (1025, 257, 24, 128, 200, F16, BF16, "mixed"),
    (520, 2051, 4160, 48, 600, BF16, BF16, "mixed"),
])
def test_adapters_against_the_formula(g, M, N, K, R, L, din, dout, ids):
    t = _inputs(M, N, K, R, L, TD[din], ids, seed=M + N + K)
    Y = _run(g, t, TD[dout])
    assert g.device_status()[0] == 0
    want, tau = _expect(t)
    _check(Y, want, tau, dout)


# Where the paths meet: a small pool beside a wide product (tiles from 129 rows on), the same
# rows with one adapter more, sorted and mixed batches of few groups, products cut along K.
@pytest.mark.parametrize("M,N,K,R,L,din,dout,ids", [
    (129, 10248, 136, 24, 8, BF16, BF16, "mixed"),
    (300, 5130, 328, 64, 8, BF16, F32, "runs"),
    (300, 5130, 328, 64, 9, BF16, F32, "runs"),
    (512, 5128, 200, 128, 4, F16, F16, "mixed"),
    (512, 264, 512, 16, 3, BF16, BF16, "runs"),
    (511, 136, 520, 40, 2, F16, BF16, "mixed"),
    (385, 130, 264, 16, 1, BF16, F32, "one"),
    (40, 600, 4096, 32, 40, BF16, F32, "mixed"),
    (90, 130, 16384, 16, 5, BF16, BF16, "mixed"),
    (600, 520, 4096, 16, 4, BF16, BF16, "mixed"),
    (520, 200, 12288, 32, 3, F16, F32, "runs"),
    # rows of Y that begin at any 2 or 4 bytes, one row, tiles of the product cut in two
    (1, 1003, 2048, 16, 3, BF16, F32, "one"),
    (1, 30, 264, 16, 3, F16, F16, "one"),
    (17, 4099, 4096, 64, 6, BF16, F32, "mixed"),
    (140, 10241, 8192, 16, 20, F16, F32, "mixed"),
    (64, 6145, 8192, 128, 9, BF16, BF16, "runs"),
    (500, 2306, 1544, 32, 1, BF16, F16, "one"),
    (2600, 2653, 200, 16, 17, F16, F16, "runs"),
    # more rows of a large pool, and past them tiles with more adapters than one group holds
    (513, 264, 520, 16, 33, BF16, BF16, "runs"),
    (2048, 130, 264, 64, 40, F16, F32, "mixed"),
    (1500, 1001, 136, 8, 700, BF16, BF16, "mixed"),
    (2049, 300, 4104, 16, 40, BF16, BF16, "mixed"),
    (2050, 257, 24, 128, 200, F16, BF16, "mixed"),
    (2100, 513, 1032, 48, 600, BF16, BF16, "mixed"),
])
def test_adapters_around_the_choice_of_path(g, M, N, K, R, L, din, dout, ids):
    t = _inputs(M, N, K, R, L, TD[din], ids, seed=13 * M + N + K)
    want, tau = _expect(t)
    _check(_run(g, t, TD[dout]), want, tau, dout)


def test_every_rank(g):
    for R in range(8, 129, 8):
        t = _inputs(150, 264, 520, R, 6, torch.bfloat16, "mixed", seed=R, scale=False)
        want, tau = _expect(t)
        _check(_run(g, t, torch.bfloat16), want, tau, BF16)


def test_same_result_every_time_and_on_another_stream(g):
    for M in (256, 1500):
        t = _inputs(M, 1000, 4096, 16, 30, torch.bfloat16, "mixed", seed=3)
        first = _run(g, t, torch.bfloat16)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            again = _run(g, t, torch.bfloat16, stream=s)
            s.synchronize()
            assert torch.equal(first, again)


@pytest.mark.parametrize("M", [200, 900])
@pytest.mark.parametrize("where", ["down", "up", "X"])
def test_infinities_and_nan_stay_with_the_rows_that_name_them(g, M, where):
    t = _inputs(M, 300, 256, 16, 8, torch.bfloat16, "mixed", seed=11)
    clean = _run(g, t, torch.bfloat16)
    if where == "X":
        t["X"][5, 7] = float("inf")
        t["X"][9, 3] = float("nan")
        hit = torch.zeros(M, dtype=torch.bool)
        hit[[5, 9]] = True
    else:
        t[where][3, 0, 0] = float("inf")
        t[where][5, 1, 2] = float("nan")
        hit = (t["ids"] == 3) | (t["ids"] == 5)
    got = _run(g, t, torch.bfloat16)
    assert torch.equal(got.cpu()[~hit], clean.cpu()[~hit])
    if where == "X":
        assert not torch.isfinite(got.cpu()[hit]).any()
    elif where == "up":  # column 0 of adapter 3's rows, column 1 of adapter 5's
        assert not torch.isfinite(got.cpu()[t["ids"] == 3][:, 0]).any()
        assert torch.isnan(got.cpu()[t["ids"] == 5][:, 1]).all()
        assert torch.isfinite(got.cpu()[:, 2:]).all()


def test_large_and_small_intermediate_values_in_fp16(g):
    # Down x up to 2^18 and down to 2^-30: outside fp16, which u must not be squeezed into
    gen = torch.Generator().manual_seed(2)
    for M in (40, 1500):
        t = _inputs(M, 264, 512, 16, 4, torch.float16, "mixed", seed=5)
        t["down"][0] *= 2.0 ** 12
        t["X"][:, :] = torch.randint(-8, 9, t["X"].shape, generator=gen).half()
        t["up"][0] = (t["up"][0].float() * 2.0 ** -10).half()
        t["down"][1] = (t["down"][1].float() * 2.0 ** -12).half()
        want, tau = _expect(t)
        _check(_run(g, t, torch.float16), want, tau, F16)


def test_row_adapter_out_of_range_is_reported_and_not_followed(g):
    for M in (50, 1500):
        t = _inputs(M, 200, 256, 16, 4, torch.bfloat16, "mixed", seed=8)
        t["ids"][3], t["ids"][10] = 4, 2 ** 31 - 1
        t["ids"][11] = -2 ** 31
        Y = _run(g, t, torch.bfloat16)
        code, word = g.device_status()
        assert code == 6 and word >> 24 == 2 and (word >> 16) & 0xFF == 1
        assert g.device_status() == (0, 0)
        want, tau = _expect(t)
        _check(Y, want, tau, BF16)


def test_captured_graph_serves_another_batch(g):
    t = _inputs(100, 520, 1024, 16, 20, torch.bfloat16, "mixed", seed=21)
    d = {k: v.cuda() for k, v in t.items()}
    Y = torch.empty(100, 520, dtype=torch.bfloat16, device="cuda")

    def call():
        g.run_adapters(d["X"], d["W"], Y, d["down"], d["up"], d["ids"], scale=d["scale"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    t["ids"] = torch.randint(-1, 20, (100,), dtype=torch.int32)
    d["ids"].copy_(t["ids"])
    graph.replay()
    torch.cuda.synchronize()
    want, tau = _expect(t)
    _check(Y, want, tau, BF16)


@pytest.mark.parametrize("M", [100, 1500])
def test_stalled_wait_times_out_and_the_next_call_is_right(M):
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    t = _inputs(M, 520, 1024, 16, 6, torch.bfloat16, "mixed", seed=31)
    want, tau = _expect(t)
    with Gemm() as g:
        _run(g, t, torch.bfloat16)
        g.set_wait_limit(50_000_000)          # 50 ms
        g.set_test_stall(True)
        _run(g, t, torch.bfloat16)
        code, word = g.device_status()
        assert code == 5 and word >> 24 == 1, (code, hex(word))
        g.set_test_stall(False)
        g.set_wait_limit(2_000_000_000)
        _check(_run(g, t, torch.bfloat16), want, tau, BF16)
        assert g.device_status() == (0, 0)


def test_forced_configurations(g):
    from dense_gemm_blackwell_02_gb300.binding import GemmError
    few = _inputs(100, 520, 1024, 16, 6, torch.bfloat16, "mixed", seed=32)
    many = _inputs(700, 520, 1024, 16, 6, torch.bfloat16, "mixed", seed=33)
    try:
        for cfg in (dict(variant=1), dict(splits=3), dict(variant=2, max_ctas=10)):
            g.set_config(**cfg)
            want, tau = _expect(few)
            _check(_run(g, few, torch.bfloat16), want, tau, BF16)
        for cfg in (dict(splits=3), dict(splits=-1), dict(group_m=1), dict(max_ctas=6),
                    dict(chain_kblocks=3)):
            g.set_config(**cfg)
            want, tau = _expect(many)
            _check(_run(g, many, torch.bfloat16), want, tau, BF16)
        for cfg in (dict(variant=1), dict(block_n=128), dict(epilogue=2), dict(swap_ab=2)):
            g.set_config(**cfg)
            with pytest.raises(GemmError, match="UNSUPPORTED"):
                _run(g, many, torch.bfloat16)
    finally:
        g.reset_config()


def test_empty_and_degenerate_calls(g):
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    dev = "cuda"
    X = torch.randn(5, 64, device=dev).bfloat16()
    W = torch.randn(40, 64, device=dev).bfloat16()
    Y = torch.empty(5, 40, dtype=torch.bfloat16, device=dev)
    ids = torch.zeros(5, dtype=torch.int32, device=dev)
    e = torch.empty
    # an empty pool: the product itself
    g.run_adapters(X, W, Y, e(0, 8, 64, dtype=X.dtype, device=dev), e(0, 40, 8, dtype=X.dtype, device=dev),
                   torch.full_like(ids, -1))
    C = torch.empty_like(Y)
    g.run(X, W, C)
    assert torch.equal(C, Y)
    # no rows, no columns: nothing happens
    g.run_adapters(X[:0], W, Y[:0], e(2, 8, 64, dtype=X.dtype, device=dev),
                   e(2, 40, 8, dtype=X.dtype, device=dev), ids[:0])
    # K = 0 writes zeros
    Y.fill_(1)
    g.run_adapters(X[:, :0].contiguous(), W[:, :0].contiguous(), Y, e(2, 8, 0, dtype=X.dtype, device=dev),
                   e(2, 40, 8, dtype=X.dtype, device=dev), ids)
    assert (Y == 0).all()


def test_refusals(g):
    from dense_gemm_blackwell_02_gb300.binding import GemmError
    dev = "cuda"
    X = torch.zeros(5, 64, device=dev, dtype=torch.bfloat16)
    W = torch.zeros(40, 64, device=dev, dtype=torch.bfloat16)
    Y = torch.zeros(5, 40, dtype=torch.bfloat16, device=dev)
    ids = torch.zeros(5, dtype=torch.int32, device=dev)

    def pool(L, R, N=40, K=64, dt=torch.bfloat16):
        return torch.zeros(L, R, K, dtype=dt, device=dev), torch.zeros(L, N, R, dtype=dt, device=dev)
    for R in (4, 12, 136):
        with pytest.raises(GemmError, match="UNSUPPORTED"):
            g.run_adapters(X, W, Y, *pool(2, R), ids)
    with pytest.raises(ValueError, match="row_adapter"):
        g.run_adapters(X, W, Y, *pool(2, 8), ids.long())
    with pytest.raises(ValueError, match="row_adapter"):
        g.run_adapters(X, W, Y, *pool(2, 8), ids[:4])
    with pytest.raises(ValueError, match="up"):
        g.run_adapters(X, W, Y, pool(2, 8)[0], pool(2, 8, N=39)[1], ids)
    with pytest.raises(ValueError, match="down"):
        g.run_adapters(X, W, Y, *pool(2, 8, dt=torch.float16), ids)
    with pytest.raises(ValueError, match="scale"):
        g.run_adapters(X, W, Y, *pool(2, 8), ids, scale=torch.ones(3, device=dev))
    with pytest.raises(ValueError, match="W must"):
        g.run_adapters(X, W[:, :56], Y, *pool(2, 8), ids)
    with pytest.raises(ValueError, match="Y must"):
        g.run_adapters(X, W, Y[:, ::2], *pool(2, 8), ids)
    odd = torch.zeros(5, 60, device=dev, dtype=torch.bfloat16)
    with pytest.raises(GemmError, match="UNSUPPORTED"):
        g.run_adapters(odd, torch.zeros(40, 60, device=dev, dtype=torch.bfloat16), Y, *pool(2, 8, K=60), ids)
    with pytest.raises(GemmError, match="UNSUPPORTED"):
        g.run_adapters(X.float(), W.float(), Y, *pool(2, 8, dt=torch.float32), ids)
    flat = torch.zeros(2 * 8 * 64 + 1, dtype=torch.bfloat16, device=dev)
    with pytest.raises(GemmError, match="UNSUPPORTED"):
        g.run_adapters(X, W, Y, flat[1:].view(2, 8, 64), pool(2, 8)[1], ids)
    assert g.device_status()[0] == 0
