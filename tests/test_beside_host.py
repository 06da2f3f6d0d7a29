"""Which product runs beside the adapters' kernels for few rows, on the host side alone."""
import pytest

from tests.fake_cuda import Fake


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    return Fake(tmp_path_factory.mktemp("fake"))


def _product(fake, M, N, K, rank=16, count=16):
    """(kernel's name, CTAs) of the call's first launch."""
    h = fake.create()
    fake.journal()
    assert fake.run_adapters(h, M, N, K, rank, count) == 0
    name, ctas = next((name, n) for w, _, n, _, name in fake.journal() if w == "launch")
    fake.lib.gemm_destroy(h)
    return name, ctas


@pytest.mark.parametrize("N,K,tiles", [
    (5120, 8192, True), (6144, 8192, True), (7168, 8192, True), (8192, 8192, True), (10240, 4096, True),
    (10240, 2048, True), (28672, 1024, True), (1024, 14336, True), (2048, 14336, True),
    (1024, 8192, False), (2048, 2048, False), (4096, 4096, False), (4096, 8192, False),
    (7168, 4096, False), (8192, 1024, False)])
def test_one_row_takes_the_form_that_measured_faster(fake, N, K, tiles):
    name, _ = _product(fake, 1, N, K, count=8)
    assert ("gemv" not in name) == tiles, name


def test_a_long_product_keeps_its_slices_where_narrow_tiles_could_have_none(fake):
    # 80 tiles of 128 x 128 leave no SM for a second slice: K 16384 in one piece took 68 us, in
    # the slices of wider tiles 53
    assert _product(fake, 256, 5120, 16384)[1] >= 100
    # where the tiles leave room, or K is short, they are taken
    for M, N, K in ((16, 512, 8192), (64, 1024, 4096), (256, 1024, 4096), (256, 512, 1024)):
        name, ctas = _product(fake, M, N, K)
        assert "ILi1ELi128" in name, name
