"""Which strides gemm_rotary takes, on the host side alone."""
import itertools
import random

import pytest

from tests.fake_cuda import Fake


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    return Fake(tmp_path_factory.mktemp("fake"))


@pytest.fixture(scope="module")
def h(fake):
    h = fake.create()
    yield h
    fake.lib.gemm_destroy(h)


def _overlaps(tokens, heads, dim, stride):
    starts = sorted(t * stride[0] + i * stride[1] for t, i in itertools.product(range(tokens), range(heads)))
    return any(b - a < dim for a, b in zip(starts, starts[1:]))


def test_a_result_whose_heads_overlap_is_refused(fake, h):
    # (several threads would write one element, in place also read it)
    fake.journal()
    for T, H, y in ((5, 3, (0, 8)), (5, 3, (24, 0)), (5, 1, (0, 8)), (1, 3, (24, 0)), (5, 3, (8, 8)),
                    (5, 3, (24, 7)), (5, 3, (4, 100)), (8, 7, (48, 56))):
        assert fake.rotary(h, T, H, 8, (1000, 100), y) == 1, (T, H, y)
        assert fake.rotary(h, T, H, 8, y, y, in_place=True) == 1, (T, H, y)
    assert not [w for w, *_ in fake.journal() if w == "launch"]
    # x may: it is only read
    assert fake.rotary(h, 5, 3, 8, (0, 8), (24, 8)) == 0
    assert fake.rotary(h, 5, 3, 8, (24, 0), (24, 8)) == 0


def test_every_stride_without_an_overlap_is_taken(fake, h):
    rng = random.Random(3)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        T, H, D = rng.randint(1, 9), rng.randint(1, 9), rng.choice([8, 9, 16])
        y = (rng.randint(0, 200), rng.randint(0, 200))
        bad = _overlaps(T, H, D, y)
        seen[bad] += 1
        assert fake.rotary(h, T, H, D, (1000, 100), y) == (1 if bad else 0), (T, H, D, y)
    assert min(seen.values()) > 300


def test_strides_of_a_single_token_or_head_do_not_count(fake, h):
    assert fake.rotary(h, 1, 3, 8, (77, 8), (5, 8), in_place=True) == 0
    assert fake.rotary(h, 5, 1, 8, (16, 77), (16, 0), in_place=True) == 0
    assert fake.rotary(h, 5, 1, 8, (16, 77), (24, 77), in_place=True) == 1


def test_large_strides_and_counts_are_checked_quickly(fake, h):
    import time
    t0 = time.perf_counter()
    assert fake.rotary(h, 40000, 50000, 8, (400000, 8), (400000, 8)) == 0
    assert fake.rotary(h, 40000, 50000, 8, (8, 320000), (8, 320000)) == 0
    assert fake.rotary(h, 40000, 50000, 8, (400000, 8), (399999, 8)) == 1
    assert time.perf_counter() - t0 < 0.1
