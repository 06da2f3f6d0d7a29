"""Normed heads and their gradients refuse results that overlap an input or another result, whatever
the strides, and nothing else: the checks against every byte's place, without a GPU."""
import random

import pytest

from tests.test_layer_host import A, fake, h  # noqa: F401

SIZE = 2  # bytes of an element


def _norm(fake, h, T, H, D, x, y, sx, sy, tables=None):  # noqa: F811
    from dense_gemm_blackwell_02_gb300.binding import _NORM_ROTARY_CALL
    t = {"wq": A[5], "wk": A[6], "cos": A[2], "sin": A[3], "pos": A[4], **(tables or {})}
    return fake.lib.gemm_norm_rotary_packed(_NORM_ROTARY_CALL.pack(
        h.value, x, y, T, H, D, *sx, *sy, 0, t["wq"], t["wk"], 2, 1, 1e-6, t["cos"], t["sin"], t["pos"], 0, 100, 1, 2, 0,
        0, 1, 0))


def _grad(fake, h, T, H, D, x, dy, dx, sx, sg, sd, dq=A[8], dk=A[9], tables=None):  # noqa: F811
    from dense_gemm_blackwell_02_gb300.binding import _NORM_ROTARY_GRAD_CALL
    t = {"wq": A[5], "wk": A[6], "cos": A[2], "sin": A[3], "pos": A[4], **(tables or {})}
    return fake.lib.gemm_norm_rotary_grad_packed(_NORM_ROTARY_GRAD_CALL.pack(
        h.value, x, dy, dx, T, H, D, *sx, *sg, *sd, 0, t["wq"], t["wk"], 2, 1, 1e-6, t["cos"], t["sin"], t["pos"], 0, 100,
        1, 2, 0, 0, dq, dk, 1, 0))


def _places(at, T, H, D, s):
    return {at + SIZE * (t * s[0] + i * s[1] + d) for t in range(T) for i in range(H) for d in range(D)}


def _launches(fake):  # noqa: F811
    return [w for w, *_ in fake.journal() if w == "launch"]


def test_results_of_every_layout_against_every_place(fake, h):  # noqa: F811
    rng = random.Random(7)
    seen = {0: 0, 1: 0}
    for _ in range(6000):
        T, H, D = rng.randint(1, 5), rng.randint(1, 4), rng.choice([2, 3, 4])

        def strides(like=None):
            if like is not None and rng.random() < 0.4:
                return like
            kind = rng.randrange(4)
            if kind == 0:                                # rows of heads, wider or not
                return (H * D + rng.choice([0, 0, D, 7]), D)
            if kind == 1:                                # heads first
                return (D, T * D + rng.choice([0, 3]))
            if kind == 2:                                # every second head
                return (2 * H * D, 2 * D)
            return (rng.randint(0, 40), rng.randint(0, 40))
        sy = strides()
        py = [sy[0] * t + sy[1] * i + d for t in range(T) for i in range(H) for d in range(D)]
        if len(set(py)) < len(py):                       # (refused for itself)
            continue
        sx, sg = strides(sy), strides(sy)
        base = 1 << 40
        y, x, dy = (base + SIZE * rng.randint(-30, 30) for _ in range(3))
        if rng.random() < 0.2:
            x = y
        if rng.random() < 0.2:
            dy = y
        mine = _places(y, T, H, D, sy)

        def same(a, b):
            return (T == 1 or a[0] == b[0]) and (H == 1 or a[1] == b[1])
        bad = bool(mine & _places(x, T, H, D, sx)) if x != y else not same(sx, sy)
        assert _norm(fake, h, T, H, D, x, y, sx, sy) == int(bad), (T, H, D, x - y, sx, sy)
        seen[int(bad)] += 1
        bad = bool(mine & _places(x, T, H, D, sx)) or (bool(mine & _places(dy, T, H, D, sg)) if dy != y
                                                       else not same(sg, sy))
        assert _grad(fake, h, T, H, D, x, dy, y, sx, sg, sy) == int(bad), (T, H, D, x - y, dy - y, sx, sg, sy)
        seen[int(bad)] += 1
    assert min(seen.values()) > 1000, seen
    fake.journal()


def test_heads_that_begin_inside_others(fake, h):  # noqa: F811
    fake.journal()
    T, H, D = 8192, 64, 128
    wide = ((H + 8) * D, D)
    for shift in (D, -D, 1, 8 * wide[0], 63 * D):
        assert _norm(fake, h, T, H, D, A[0], A[0] + SIZE * shift, wide, wide) == 1, shift
        assert _grad(fake, h, T, H, D, A[0], A[1], A[0] + SIZE * shift, wide, wide, wide) == 1, shift
        assert _grad(fake, h, T, H, D, A[0], A[1], A[1] + SIZE * shift, wide, wide, wide) == 1, shift
    assert not _launches(fake)
    # heads of one fused row beside each other, and what only touches, are no overlap
    fused = (3 * H * D, D)
    for shift in (H * D, 2 * H * D, -H * D):
        assert _norm(fake, h, T, H, D, A[0], A[0] + SIZE * shift, fused, fused) == 0, shift
        assert _grad(fake, h, T, H, D, A[0], A[0] + SIZE * H * D, A[0] + 2 * SIZE * H * D, fused, fused, fused) == 0
    assert _norm(fake, h, T, H, D, A[0], A[0] + SIZE * T * H * D, (H * D, D), (H * D, D)) == 0
    # every second of a row's 192 heads, from number 64 to 190, and from 62 on
    assert _norm(fake, h, T, H, D, A[0], A[0] + SIZE * H * D, fused, (3 * H * D, 2 * D)) == 0
    assert _norm(fake, h, T, H, D, A[0], A[0] + SIZE * (H - 2) * D, fused, (3 * H * D, 2 * D)) == 1
    assert _norm(fake, h, 1 << 20, H, D, A[0], A[0] + SIZE * H * D, (1 << 40, D), (1 << 40, D)) == 0


@pytest.mark.parametrize("name,nbytes", [("wq", 512), ("wk", 512), ("cos", 400), ("sin", 400), ("pos", 20)])
def test_results_inside_what_is_read(fake, h, name, nbytes):  # noqa: F811
    fake.journal()
    T, H, D = 5, 3, 128
    s = (H * D, D)
    at = {"wq": A[5], "wk": A[6], "cos": A[2], "sin": A[3], "pos": A[4]}[name]
    for place in (at, at + nbytes - 4, at - SIZE * T * H * D + 4):
        assert _norm(fake, h, T, H, D, A[0], place, s, s) == 1
        assert _grad(fake, h, T, H, D, A[0], A[1], place, s, s, s) == 1
    for place in (at, at + nbytes - 4, at - 512 + 4):
        assert _grad(fake, h, T, H, D, A[0], A[1], A[7], s, s, s, dq=place) == 1
        assert _grad(fake, h, T, H, D, A[0], A[1], A[7], s, s, s, dk=place) == 1
    assert not _launches(fake)
    assert _norm(fake, h, T, H, D, A[0], at + nbytes, s, s) == 0
    assert _grad(fake, h, T, H, D, A[0], A[1], A[7], s, s, s, dq=at + nbytes, dk=at - 512) == 0


def test_weights_gradients_inside_each_other_and_the_heads(fake, h):  # noqa: F811
    fake.journal()
    T, H, D = 5, 3, 128
    s = (2 * H * D, D)
    for dk in (A[8] + 4 * (D - 1), A[8] - 4 * (D - 1), A[8] + 4):
        assert _grad(fake, h, T, H, D, A[0], A[1], A[7], s, s, s, dk=dk) == 1
    for t in (A[0], A[1], A[7]):
        for place in (t, t + SIZE * (2 * H * D) + 4, t - 4 * D + 4, t + SIZE * (4 * 2 * H * D + H * D) - 4):
            assert _grad(fake, h, T, H, D, A[0], A[1], A[7], s, s, s, dq=place) == 1
            assert _grad(fake, h, T, H, D, A[0], A[1], A[7], s, s, s, dk=place) == 1
    assert not _launches(fake)
    # between the tokens' heads there is room
    assert _grad(fake, h, T, H, D, A[0], A[1], A[7], s, s, s, dq=A[7] + SIZE * H * D, dk=A[0] + SIZE * 3 * H * D) == 0
    assert _grad(fake, h, T, H, D, A[0], A[1], A[7], s, s, s, dk=A[8] + 4 * D) == 0
    assert _grad(fake, h, T, H, D, A[0], A[1], A[7], s, s, s, dq=0, dk=0) == 0
