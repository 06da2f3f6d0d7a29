"""The handle's device memory, on the host side alone: how it is cleared, grown and kept."""
import pytest

from tests.fake_cuda import Fake

STREAM = 0x7770


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    return Fake(tmp_path_factory.mktemp("fake"))


def _sizes(journal, what):
    return {p: n for w, p, n, _, _ in journal if w == what}


def _cleared_in_time(journal):
    """Whether every clear before a launch is done by then: queued on the launch's own
    stream, or on another that was waited for."""
    pending = set()
    for what, _, _, stream, name in journal:
        if what == "memset":
            pending.add((stream, "legacy" in name))
        elif what == "synchronize":
            pending = {p for p in pending if p[0] != stream or p[1]}
        elif what == "synchronize-device":
            pending = set()
        elif what == "launch":
            assert not pending - {(stream, False)}, f"{name} may run before {pending} are cleared"


@pytest.mark.parametrize("call", ["few", "many", "split"])
def test_counters_are_cleared_before_the_first_kernel_of_a_new_handle(fake, call):
    # the groups' counters (few), the product's arrival counters (many, cut along K; split)
    fake.journal()
    h = fake.create()
    if call == "split":
        assert fake.run(h, 256, 1000, 16384, STREAM) == 0
    else:
        assert fake.run_adapters(h, *((64, 512, 512) if call == "few" else (600, 1000, 8192)), 16, 4, STREAM) == 0
    journal = fake.journal()
    assert sum(w == "launch" for w, *_ in journal) == {"few": 3, "many": 2, "split": 1}[call]
    assert sum(w == "memset" for w, *_ in journal) >= 1
    _cleared_in_time(journal)
    fake.lib.gemm_destroy(h)


def test_memory_of_earlier_calls_outlives_the_handles_growth(fake):
    # (a graph that was captured at the smaller sizes names it)
    fake.journal()
    h = fake.create()
    for call in ("run_adapters", "run"):
        for rows in (8, 64, 200, 500, 600, 2000, 8000):
            sizes = (rows, 1000, 8192) + ((16, 4) if call == "run_adapters" else ())
            assert getattr(fake, call)(h, *sizes) == 0
    journal = fake.journal()
    assert not _sizes(journal, "free")
    made = _sizes(journal, "malloc")
    assert len(made) >= 6                               # it did grow, workspace and counters alike
    fake.lib.gemm_destroy(h)
    assert _sizes(fake.journal(), "free") == made


def test_growing_in_small_steps_keeps_little(fake):
    fake.journal()
    h = fake.create()
    for rows in range(1, 513):
        assert fake.run_adapters(h, rows, 1000, 4096, 16, 40) == 0
    made = _sizes(fake.journal(), "malloc")
    need = 512 * (1000 * 4 + 16 * 16 * 4 + 128) + 1024  # the largest call's scratch
    assert len(made) < 32 and sum(made.values()) < 4 * need + 40 * 2 ** 20  # (and the product's)
    fake.lib.gemm_destroy(h)


def test_memory_that_cannot_double_grows_to_what_is_needed_or_stays(fake):
    h = fake.create()
    assert fake.run_adapters(h, 100, 1000, 512, 16, 4) == 0
    fake.journal()
    try:
        fake.lib.fake_largest(700 * 1024)               # twice the first call's does not fit
        assert fake.run_adapters(h, 120, 1000, 512, 16, 4) == 0
        grown = _sizes(fake.journal(), "malloc")
        assert grown and all(n < 700 * 1024 for n in grown.values())
        assert fake.run_adapters(h, 400, 1000, 512, 16, 4) == 4  # GEMM_ERR_OOM, nothing queued
        assert not [w for w, *_ in fake.journal() if w in ("launch", "free")]
    finally:
        fake.lib.fake_largest(2 ** 63)
    assert fake.run_adapters(h, 120, 1000, 512, 16, 4) == 0
    assert not _sizes(fake.journal(), "malloc")
    fake.lib.gemm_destroy(h)


def test_an_aborted_run_has_every_counter_cleared(fake):
    import ctypes
    fake.journal()
    h = fake.create()
    assert fake.run(h, 256, 1000, 16384) == 0 and fake.run(h, 600, 1000, 8192) == 0
    assert fake.run_adapters(h, 64, 512, 512, 16, 4) == 0
    journal = fake.journal()
    cleared = _sizes(journal, "memset")                 # status word and counters, when made
    assert len(cleared) >= 4
    status = next(p for w, p, *_ in journal if w == "memset")
    ctypes.c_uint32.from_address(status).value = 1 << 24
    assert fake.lib.gemm_device_status(h, None, None) == 5
    assert _sizes(fake.journal(), "memset") == cleared
    fake.lib.gemm_destroy(h)


def test_counters_are_zero_again_after_a_launch_that_fails(fake):
    # (few_down has listed its groups, and few_up, which clears the list's length, never runs)
    fake.journal()
    h = fake.create()
    try:
        assert fake.run_adapters(h, 64, 512, 512, 16, 4, STREAM) == 0
        journal = fake.journal()
        counters = [p for w, p, n, *_ in journal if w == "memset" and n == 8]
        assert len(counters) == 1
        fake.lib.fake_fail(b"few_up_kernel")
        assert fake.run_adapters(h, 64, 512, 512, 16, 4, STREAM) == 3  # GEMM_ERR_CUDA
        after = fake.journal()
        at = [w for w, *_ in after].index("failed-launch")
        assert [(w, p, n, s) for w, p, n, s, _ in after[at + 1:]] == [("memset", counters[0], 8, STREAM)]
        fake.lib.fake_fail(b"few_down_kernel")
        assert fake.run_adapters(h, 64, 512, 512, 16, 4, STREAM) == 3
    finally:
        fake.lib.fake_fail(b"")
    assert fake.run_adapters(h, 64, 512, 512, 16, 4, STREAM) == 0
    fake.lib.gemm_destroy(h)
