"""Host side of the gated block's gradients in fp16: which kernels are queued, and the memory that is
zero between calls."""
from tests.test_layer_host import A, _gated_grad, fake, h  # noqa: F401

KERNELS = ("slope_range", "slope_scale", "pair", "rank", "join")


def _order(fake, call, code=0):  # noqa: F811
    fake.journal()
    assert call() == code
    return [next(k for k in KERNELS if f"gated_{k}_kernel" in name) for w, _, _, _, name in fake.journal(clear=False)
            if w == "launch"]


def test_launches_in_fp16(fake, h):  # noqa: F811
    def order(*size, **kw):
        return _order(fake, lambda: _gated_grad(fake, h, *size, dtype=0, **kw))
    assert order(1025, 1401, 2008) == ["slope_range", "slope_scale", "pair"]
    assert order(100, 14336, 4096) == ["slope_range", "slope_scale", "pair", "join"]
    assert order(8, 500, 512) == ["rank", "slope_range", "slope_scale", "pair"]
    assert order(8, 14336, 4096, dX=0, Wg=0, Wu=0) == ["rank"]
    assert order(300, 4096, 4096, dX=0, Wg=0, Wu=0) == ["slope_range", "slope_scale", "pair"]
    assert order(300, 4096, 4096, dWg=0, dWu=0, X=0) == ["slope_range", "slope_scale", "pair"]


def test_largest_magnitudes_start_from_zero(fake):  # noqa: F811
    # (a handle of its own: its memory is seen to grow)
    h = fake.create()
    fake.journal()
    M, N, K = 301, 520, 264
    assert _gated_grad(fake, h, M, N, K, dtype=0) == 0
    rows = fake.journal()
    scratch = [n for w, _, n, _, _ in rows if w == "malloc"]
    words = 304 + 2 * N                                  # rows in whole fours, and both columns
    assert 4 * words in scratch                          # what is zero between calls
    assert max(scratch) >= 8 * M * N + 4 * words         # two copies of dG and dU, the scales
    assert [n for w, _, n, _, _ in rows if w == "memset"] == [4 * words]
    # a second call finds it as the first one's products left it
    assert _gated_grad(fake, h, M, N, K, dtype=0) == 0
    assert [w for w, *_ in fake.journal() if w in ("memset", "malloc")] == []
    # products that were not queued leave nothing: it is cleared on the stream
    fake.lib.fake_fail(b"gated_pair_kernel")
    assert _gated_grad(fake, h, M, N, K, dtype=0) != 0
    fake.lib.fake_fail(b"")
    assert [n for w, _, n, _, _ in fake.journal() if w == "memset"] == [4 * words]
    # bf16 has no such memory
    other = fake.create()
    fake.journal()
    assert _gated_grad(fake, other, M, N, K, dtype=1) == 0
    assert [w for w, *_ in fake.journal() if w == "memset"] == []
    for x in (h, other):
        fake.lib.gemm_destroy(x)
