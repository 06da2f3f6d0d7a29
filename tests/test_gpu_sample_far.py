"""The choice of the next token (gemm_sample) from peaked rows, whose other tokens have weights of
2^-40 and less, and at the ends of the random numbers' range, where such a token is the answer: the
first that stays at 0 and below (and for NaN), the last that stays from 1 on.  Reference and
tolerances as in test_gpu_sample: tokens have to be equal, and weights below 2^-60 count as 0."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_sample import DT, _check, _logits, _row, g  # noqa: F401

pytestmark = pytest.mark.gpu

ENDS = [0.0, -1.0, float("nan"), 1 - 2.0 ** -24, 1.0, 2.0, float("inf")]
# log2 of the other tokens' weights: below and above a 2^-43rd, next to 2^-60, and beyond it
DEPTHS = [40.3, 42.8, 44.7, 50.2, 59.5, 61.0]


def _peaked(V, depth, largest, dt):
    z = torch.full((V,), -depth * math.log(2.0))
    z[largest] = 0.0
    return z.to(DT[dt])


def _rows(V, dt):
    """Every depth with every random number, the largest logit last (random below 0.5) or first."""
    z, u = [], []
    for depth in DEPTHS:
        for r in ENDS:
            z.append(_peaked(V, depth, 0 if r > 0.5 else V - 1, dt))
            u.append(r)
    return torch.stack(z), torch.tensor(u)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("V", [300, 5003, 128256])
def test_peaked_rows_at_the_ends_of_the_random_numbers(g, dt, V):  # noqa: F811
    z, u = _rows(V, dt)
    B = len(u)
    _check(g, z, u)
    for i in range(0, B, 5):                             # one row, spread over a cluster
        _check(g, z[i:i + 1], u[i:i + 1])
    _check(g, z, u, top_k=torch.full((B,), 5).int())
    _check(g, z, u, top_k=torch.full((B,), V - 1).int())
    _check(g, z, u, top_k=torch.full((B,), V // 2).int())
    _check(g, z, u, min_p=torch.full((B,), 2.0 ** -47))
    _check(g, z, u, top_p=torch.full((B,), 0.9))
    _check(g, z, u, top_k=torch.full((B,), V - 2).int(), top_p=torch.full((B,), 0.9), min_p=torch.full((B,), 2.0 ** -47))


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_tails_of_many_depths(g, dt):  # noqa: F811
    """The others' weights spread from 2^-26 to 2^-66: what is behind 2^-60 never stays, what is in
    front of it does."""
    gen = torch.Generator().manual_seed(12)
    V, B = 40007, len(ENDS)
    z = (-(26 + 40 * torch.rand(B, V, generator=gen)) * math.log(2.0)).to(DT[dt])
    z[:, V // 2] = 0.0
    # (no weight may lie next to the 2^-60 that decides whether it counts)
    far = (-z.double() / math.log(2.0) - 60).abs() < 2.0 ** -10
    z[far] = -100.0
    u = torch.tensor(ENDS)
    _check(g, z, u)
    for k in (3, 900, 2500, 20000):
        _check(g, z, u, top_k=torch.full((B,), k).int())
        _check(g, z, u, top_k=torch.full((B,), k).int(), min_p=torch.full((B,), 2.0 ** -58.5))
    _check(g, z, u, min_p=torch.full((B,), 2.0 ** -44.4))


def test_the_longest_peaked_rows(g):  # noqa: F811
    """2^20 logits, 31 below the largest: together 2^-24.7, which torch.rand's smallest numbers reach."""
    V = 1 << 20
    z = torch.stack([_peaked(V, 44.7, at, "f32") for at in (V - 1, 0, V // 2)])
    tokens = torch.full((3,), -7, dtype=torch.int32, device="cuda")
    for u in ENDS + [2.0 ** -24, 2.0 ** -26, 3 * 2.0 ** -27]:
        r = torch.tensor([u, u, u])
        tokens.fill_(-7)
        probs = torch.full((3,), float("nan"), device="cuda")
        g.sample(z.cuda(), tokens, r.cuda(), probs=probs)
        for i in range(3):
            want, prob, margin = _row(z[i].double().numpy(), float(r[i]))
            got = int(tokens[i])
            # a running sum within 2^-33 of the whole: 2^-33 / 2^-44.7 tokens either way
            assert abs(got - want) <= (0 if margin > 2.0 ** -33 else 2.0 ** 11.7), (u, i, got, want)
            assert abs(float(probs[i]) / prob - 1) <= 2.0 ** -24 + 2.0 ** -21 or got != want


def test_rows_of_batches_whose_draw_is_at_an_end(g):  # noqa: F811
    """More rows than run at once, a fifth of them peaked, every fourth random number at an end."""
    gen = torch.Generator().manual_seed(3)
    B, V = 320, 20011
    z = _logits(gen, B, V, "bf16")
    for i in range(0, B, 5):
        z[i] = _peaked(V, DEPTHS[i // 5 % len(DEPTHS)], int(torch.randint(0, V, (1,), generator=gen)), "bf16")
    u = torch.rand(B, generator=gen)
    u[::4] = torch.tensor([0.0, 1.0])[torch.arange(B // 4) % 2]
    _check(g, z, u)
    k = torch.tensor([0, 40, 3, 5000])[torch.arange(B) % 4].int()
    _check(g, z, u, top_k=k)
    _check(g, z, u, top_k=k, top_p=torch.tensor([1.0, 0.9])[torch.arange(B) % 2])


def test_the_reference_itself():
    """The rows' expected tokens, by hand."""
    z = _peaked(300, 44.7, 299, "f32").double().numpy()
    assert _row(z, 0.0)[0] == 0 and _row(z, 1.0)[0] == 299 and _row(z, float("nan"))[0] == 0
    z = _peaked(300, 44.7, 0, "f32").double().numpy()
    assert _row(z, 1.0)[0] == 299 and _row(z, 1 - 2.0 ** -24)[0] == 0
    assert _row(z, 1.0, k=5)[0] == 4 and _row(z, 1.0, least=2.0 ** -44)[0] == 0
    assert _row(_peaked(300, 61.0, 0, "f32").double().numpy(), 1.0)[0] == 0
    assert abs(_row(z, 1.0)[1] / 2.0 ** -44.7 - 1) < 1e-5 and np.isfinite(z).all()
