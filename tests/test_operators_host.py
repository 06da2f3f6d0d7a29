"""Host side of the operators around the projections: what is refused without a GPU, and
how sections of axes spread over the rotary pairs."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from dense_gemm_blackwell_02_gb300 import binding, build
    build.build()
    return binding.lib()


def test_null_handles_and_descriptions_are_rejected(lib):
    from dense_gemm_blackwell_02_gb300.binding import GemmAdapters, GemmLogits, GemmRotary
    ad, ro, lo = GemmAdapters(), GemmRotary(), GemmLogits()
    assert lib.gemm_run_adapters(None, None, None, None, 1, 1, 8, 0, 0, ctypes.byref(ad), None, None) == 1
    assert lib.gemm_rotary(None, None, None, 1, 1, 2, 2, 2, 2, 2, 0, ctypes.byref(ro), None) == 1
    assert lib.gemm_adjust_logits(None, None, None, 1, 1, 1, 1, 0, 0, ctypes.byref(lo), None) == 1


def test_the_status_of_a_bad_index_has_a_text(lib):
    assert b"out of range" in lib.gemm_status_string(6)


@pytest.mark.parametrize("sections,interleaved,want", [
    ([2, 1], False, [0, 0, 1]),
    ([2, 1], True, [0, 1, 0]),
    ([1, 3, 2], True, [0, 1, 2, 1, 2, 1]),
    ([0, 2], True, [1, 1]),
    ([4], True, [0, 0, 0, 0]),
])
def test_pair_axes(sections, interleaved, want):
    from dense_gemm_blackwell_02_gb300.binding import pair_axes
    assert pair_axes(sections, interleaved) == want


def test_pair_axes_refuses_what_are_no_sections():
    from dense_gemm_blackwell_02_gb300.binding import pair_axes
    for bad in ([], [3, -1]):
        with pytest.raises(ValueError):
            pair_axes(bad)
