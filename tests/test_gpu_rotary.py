"""Rotary positions with several axes (gemm_rotary) against the formula in 64 bits.

Tolerance.  a' = a cos - b sin in binary32 rounds at most three times, each within 2^-24 of
|a cos| + |b sin|, then once to the output type:  ulp / 2 + 4 * 2^-24 * (|a cos| + |b sin|).
"""
import numpy as np
import pytest
import torch

from tests import parity

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"f16": 0, "bf16": 1, "f32": 2}


@pytest.fixture(scope="module")
def g():
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    h = Gemm()
    yield h
    h.close()


def _tables(P, half):
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    ang = torch.arange(P, dtype=torch.float64)[:, None] * f
    return ang.cos().float(), ang.sin().float()


def _expect(x, cos, sin, pos, axes, neighbours, inverse):
    """(value, sum of the terms' magnitudes), both float64 arrays."""
    x = x.double().numpy()
    half = cos.shape[1]
    p = pos.numpy()[axes]                        # pairs x tokens
    ok = (p >= 0) & (p < len(cos))
    at = np.where(ok, p, 0)
    i = np.arange(half)[:, None]
    c = np.where(ok, cos.double().numpy()[at, i], 1.0).T[:, None, :]
    s = np.where(ok, sin.double().numpy()[at, i], 0.0).T[:, None, :]
    if inverse:
        s = -s
    y, mag = x.copy(), np.zeros_like(x)
    ia = slice(0, 2 * half, 2) if neighbours else slice(0, half)
    ib = slice(1, 2 * half, 2) if neighbours else slice(half, 2 * half)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia], mag[..., ib] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, mag


def _check(y, want, mag, dt):
    got = y.double().cpu().numpy()
    bound = parity.ulp_of(want, CODE[dt]) / 2 + 4 * 2.0 ** -24 * mag
    bad = np.argwhere(~(np.abs(got - want) <= bound * (1 + 1e-9)))
    assert bad.size == 0, f"{len(bad)} off, first {bad[0]}: {got[tuple(bad[0])]} for {want[tuple(bad[0])]}"


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("T,H,D,half,sections,mixed,inverse", [
    (1, 72, 128, 64, (16, 24, 24), False, False),
    (3, 5, 128, 64, (16, 24, 24), True, True),
    (37, 8, 80, 36, (10, 13, 13), False, True),     # a partial rotation
    (64, 1, 64, 32, (32,), False, False),
    (130, 3, 70, 35, (35,), False, False),          # odd numbers of pairs
    (9, 2, 66, 10, (0, 10), False, False),          # an axis without pairs
    (5, 7, 2, 1, (1,), False, False),
    (11, 9, 600, 256, (100, 56, 50, 50), True, False),
    (700, 40, 128, 64, (64,), False, True),
    (2500, 2, 256, 64, (20, 22, 22), False, False),
])
def test_rotary_against_the_formula(g, dt, neighbours, T, H, D, half, sections, mixed, inverse):
    from dense_gemm_blackwell_02_gb300.binding import pair_axes
    gen = torch.Generator().manual_seed(T * H + D)
    x = torch.randn(T, H, D, generator=gen).to(DT[dt])
    cos, sin = _tables(500, half)
    pos = torch.randint(0, 500, (len(sections), T), generator=gen, dtype=torch.int32)
    axes = pair_axes(sections, mixed)
    want, mag = _expect(x, cos, sin, pos, axes, neighbours, inverse)
    xd, y = x.cuda(), torch.full((T, H, D), float("nan"), dtype=DT[dt], device="cuda")
    g.rotary(xd, y, cos.cuda(), sin.cuda(), pos.cuda(), pair_axis=axes, neighbours=neighbours,
             inverse=inverse)
    _check(y, want, mag, dt)
    assert torch.equal(xd.cpu(), x)
    g.rotary(xd, xd, cos.cuda(), sin.cuda(), pos.cuda(), pair_axis=axes, neighbours=neighbours,
             inverse=inverse)                       # in place: the same bits
    assert torch.equal(xd, y)
    assert g.device_status()[0] == 0


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("offset,heads_first", [(0, False), (8, False), (1, False), (0, True)])
def test_heads_inside_wider_rows_and_other_orders(g, neighbours, offset, heads_first):
    T, H, D, half = 50, 6, 64, 32
    gen = torch.Generator().manual_seed(4)
    if heads_first:                                  # heads x tokens x dim in memory
        wide = torch.randn(H, T, D, generator=gen).bfloat16().cuda()
        x = wide.transpose(0, 1)
    else:
        wide = torch.randn(T, (H + 2) * D + offset, generator=gen).bfloat16().cuda()
        x = wide[:, offset:offset + H * D].unflatten(1, (H, D))
    cos, sin = _tables(100, half)
    pos = torch.randint(0, 100, (T,), generator=gen, dtype=torch.int32)
    before = wide.clone()
    want, mag = _expect(x.cpu(), cos, sin, pos[None], [0] * half, neighbours, False)
    y = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    g.rotary(x, y, cos.cuda(), sin.cuda(), pos.cuda(), neighbours=neighbours)
    _check(y, want, mag, "bf16")
    assert torch.equal(wide, before)
    g.rotary(x, x, cos.cuda(), sin.cuda(), pos.cuda(), neighbours=neighbours)
    assert torch.equal(x.contiguous(), y)
    if not heads_first:                              # what lies beside the heads is untouched
        assert torch.equal(wide[:, offset + H * D:], before[:, offset + H * D:])
        assert torch.equal(wide[:, :offset], before[:, :offset])


@pytest.mark.parametrize("neighbours", [False, True])
def test_inverse_is_the_gradient(g, neighbours):
    # y = R x is linear: for any direction d and weights w, the difference quotient of
    # <w, R x> along d is <R^T w, d>; R^T is the inverse turn.
    T, H, D, half = 40, 4, 72, 32
    gen = torch.Generator().manual_seed(9)
    cos, sin = (t.cuda() for t in _tables(300, half))
    pos = torch.randint(0, 300, (2, T), generator=gen, dtype=torch.int32).cuda()
    axes = [i % 2 for i in range(half)]
    x, d, w = (torch.randn(T, H, D, generator=gen).cuda() for _ in range(3))

    def turn(v, inverse=False):
        y = torch.empty_like(v)
        g.rotary(v, y, cos, sin, pos, pair_axis=axes, neighbours=neighbours, inverse=inverse)
        return y.double()
    eps = 0.25
    quotient = ((turn(x + eps * d) - turn(x - eps * d)) * w.double()).sum() / (2 * eps)
    grad = turn(w, inverse=True)
    inner = (grad * d.double()).sum()
    # every element of both sides is off by a few 2^-24 of numbers of size ~10; their sum of
    # T * H * D terms by at most that many times more
    assert abs(quotient - inner) <= T * H * D * 10 * 8 * 2.0 ** -24
    # and turning there and back is the identity up to the tables' cos^2 + sin^2
    back = turn(turn(x).float(), inverse=True)
    assert (back - x.double()).abs().max() <= 8 * 2.0 ** -23 * x.abs().max().double()


def test_position_out_of_range_is_reported_and_left_unturned(g):
    x = torch.randn(6, 3, 64).bfloat16()
    cos, sin = _tables(50, 32)
    pos = torch.tensor([0, 49, 50, -1, 2 ** 31 - 1, 3], dtype=torch.int32)
    y = torch.empty_like(x, device="cuda")
    g.rotary(x.cuda(), y, cos.cuda(), sin.cuda(), pos.cuda())
    code, word = g.device_status()
    assert code == 6 and word >> 24 == 2 and (word >> 16) & 0xFF == 2
    want, mag = _expect(x, cos, sin, pos[None], [0] * 32, False, False)
    _check(y, want, mag, "bf16")
    assert torch.equal(y.cpu()[2:5], x[2:5])


def test_infinities_and_nan_stay_in_their_pairs(g):
    x = torch.randn(4, 3, 64)
    cos, sin = _tables(50, 32)
    pos = torch.tensor([1, 2, 3, 4], dtype=torch.int32).cuda()
    clean, y = torch.empty(4, 3, 64, device="cuda"), torch.empty(4, 3, 64, device="cuda")
    g.rotary(x.cuda(), clean, cos.cuda(), sin.cuda(), pos)
    x[1, 2, 5], x[3, 0, 40] = float("nan"), float("inf")
    g.rotary(x.cuda(), y, cos.cuda(), sin.cuda(), pos)
    hit = torch.zeros(4, 3, 64, dtype=torch.bool)
    hit[1, 2, [5, 37]] = True
    hit[3, 0, [8, 40]] = True
    assert torch.equal(y.cpu()[~hit], clean.cpu()[~hit])
    assert not torch.isfinite(y.cpu()[hit]).any()


def test_empty_calls_and_refusals(g):
    from dense_gemm_blackwell_02_gb300.binding import GemmError
    cos, sin = (t.cuda() for t in _tables(10, 4))
    x = torch.zeros(3, 2, 8, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    g.rotary(x[:0], x[:0], cos, sin, pos[:0])
    g.rotary(x[:, :0], x[:, :0], cos, sin, pos)
    with pytest.raises(ValueError, match="positions"):
        g.rotary(x, x, cos, sin, pos[:2])
    with pytest.raises(ValueError, match="positions"):
        g.rotary(x, x, cos, sin, pos.long())
    with pytest.raises(ValueError, match="sin"):
        g.rotary(x, x, cos, sin[:, :3], pos)
    with pytest.raises(ValueError, match="pair_axis"):
        g.rotary(x, x, cos, sin, pos, pair_axis=[0, 0, 0])
    with pytest.raises(ValueError, match="pair_axis"):
        g.rotary(x, x, cos, sin, pos, pair_axis=[0, 0, 0, 1])
    with pytest.raises(ValueError, match="dtype"):
        g.rotary(x, x.half(), cos, sin, pos)
    with pytest.raises(ValueError, match="contiguous"):
        y = torch.zeros(3, 8, 2, device="cuda").transpose(1, 2)
        g.rotary(x, y, cos, sin, pos)
    wide_c, wide_s = (t.cuda() for t in _tables(10, 5))
    with pytest.raises(GemmError, match="INVALID_ARG"):
        g.rotary(x, x, wide_c, wide_s, pos)           # more pairs than the head has
    with pytest.raises(GemmError, match="INVALID_ARG"):
        y = x.as_strided((3, 2, 8), (8, 24, 1))
        g.rotary(x, y, cos, sin, pos)                 # in place with other strides
    with pytest.raises(KeyError):
        g.rotary(x.double(), x.double(), cos, sin, pos)
    assert g.device_status()[0] == 0


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("D,half", [(64, 32), (70, 35), (80, 36)])
def test_pairs_at_a_position_out_of_range_keep_infinities_and_nan(g, dt, neighbours, D, half):
    # unturned means as they are: not a * 1 - b * 0, which is NaN for an infinite b.  Pairs of
    # the other axis turn as always.
    gen = torch.Generator().manual_seed(D)
    x = torch.randn(9, 3, D, generator=gen).to(DT[dt])
    inf = float("inf")
    x[2, 1, 3], x[2, 2, 2 * half - 1], x[4, 0, 0], x[5, 1, half] = inf, -inf, float("nan"), inf
    cos, sin = _tables(50, half)
    pos = torch.tensor([[1, 49, 50, 3, -1, 2 ** 31 - 1, 0, 7, 8], [2, 3, 4, -7, 5, 6, 50, 7, 9]],
                       dtype=torch.int32)
    axes = [0] * (half // 2) + [1] * (half - half // 2)
    out_of_range = (pos < 0) | (pos >= 50)
    pair = torch.arange(half)
    a, b = (2 * pair, 2 * pair + 1) if neighbours else (pair, pair + half)
    axis = torch.zeros(D, dtype=torch.long)
    axis[a] = axis[b] = torch.tensor(axes)
    kept = out_of_range[axis].T[:, None, :].expand(9, 3, D).clone()
    kept[..., 2 * half:] = True
    y = torch.empty(9, 3, D, dtype=DT[dt], device="cuda")
    g.rotary(x.cuda(), y, cos.cuda(), sin.cuda(), pos.cuda(), pair_axis=axes, neighbours=neighbours)
    z = x.cuda()
    g.rotary(z, z, cos.cuda(), sin.cuda(), pos.cuda(), pair_axis=axes, neighbours=neighbours)
    assert g.device_status()[0] == 6
    bits = torch.int32 if dt == "f32" else torch.int16
    for got in (y.cpu(), z.cpu()):
        assert torch.equal(got.view(bits)[kept], x.view(bits)[kept])
        finite = torch.isfinite(x).all(dim=2)
        want, mag = _expect(x[finite][:, None], cos, sin, pos[:, finite.nonzero()[:, 0]], axes,
                            neighbours, False)
        _check(got[finite][:, None], want, mag, dt)
