"""The handle's device memory, on the host side alone: how it is cleared, grown and kept."""
import pytest

from tests.fake_cuda import Fake

STREAM = 0x7770


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    return Fake(tmp_path_factory.mktemp("fake"))


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
