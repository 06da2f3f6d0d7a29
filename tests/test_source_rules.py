"""Rules of the device code that no run shows reliably, checked in its source."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dense_gemm_blackwell_02_gb300", "csrc")


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def test_what_an_overlapping_kernel_writes_is_not_read_as_constant():
    # ld.global.nc (__ldg) is for memory that nothing writes while the kernel runs.  The product
    # with adapters starts while the kernel before it still writes the tiles' lists, u and its
    # factors, and few_up while few_down still writes the groups and the partial sums.
    gemm, few = _code("gemm_kernel.cuh"), _code("adapters_few_kernel.cu")
    assert "ad.tiles" in gemm and "ad.row_scale" in gemm
    for load in re.findall(r"__ldg\((?:[^()]|\([^()]*\))*\)", gemm):
        assert not re.search(r"\bad\.|\bat->", load), load
    up = few[few.index("few_up_kernel("):]
    for load in re.findall(r"__ldg\((?:[^()]|\([^()]*\))*\)", up):
        assert not re.search(r"p\.(counts|groups|partial|base)\b|entry", load), load


def test_shared_memory_that_is_read_as_a_structure_declares_its_alignment():
    # (the GEMM and the adapters' ring round their first address up themselves)
    source = _code("adapters_kernel.cu")
    assert "reinterpret_cast<TileSlots*>(smem_raw)" in source
    assert re.search(r"extern\s+__shared__\s+__align__\(16\)\s+uint8_t smem_raw", source)
