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


def test_packed_calls_reject_null_blocks_and_null_handles(lib):
    from dense_gemm_blackwell_02_gb300 import binding as b
    for call, block in ((lib.gemm_run_adapters_packed, b._ADAPTERS_CALL),
                        (lib.gemm_rotary_packed, b._ROTARY_CALL),
                        (lib.gemm_adjust_logits_packed, b._LOGITS_CALL)):
        assert call(None) == 1
        assert call(bytes(block.size)) == 1


def test_packed_blocks_have_the_headers_layout(tmp_path):
    # every field of the C structures, nested ones included, at the offset of its value in
    # the block that the binding packs
    import re
    import struct
    import subprocess
    from dense_gemm_blackwell_02_gb300 import binding as b
    adapters = ["adapters." + f for f in ("down", "up", "scale", "count", "rank")]
    rotary = ["rotary." + f for f in ("cos", "sin", "positions", "pair_axis", "num_positions", "axes",
                                      "rot_dim", "pairs", "inverse")]
    adjust = ["adjust." + n for n, _ in b.GemmLogits._fields_]
    fields = {
        "gemm_adapters_call_t": (b._ADAPTERS_CALL, "h X W Y M N K row_adapter stream dtype_in "
                                 "dtype_out".split() + adapters),
        "gemm_rotary_call_t": (b._ROTARY_CALL, "h x y tokens heads dim x_token_stride x_head_stride "
                               "y_token_stride y_head_stride stream".split() + rotary
                               + ["dtype", "axes_follow"]),
        "gemm_logits_call_t": (b._LOGITS_CALL, "h logits out rows vocab logits_stride out_stride "
                               "stream dtype_in dtype_out".split() + adjust),
    }
    lines = []
    for name, (_, names) in fields.items():
        lines += [f'printf("%zu ", offsetof({name}, {f}));' for f in names]
        lines.append(f'printf("%zu\\n", sizeof({name}));')
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "gemm.h"\n'
                   "int main(void) {" + "\n".join(lines) + "return 0; }")
    exe = tmp_path / "layout"
    import os
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.check_call(["gcc", "-I", include, str(src), "-o", str(exe)])
    out = subprocess.check_output([str(exe)], text=True).splitlines()
    for line, (block, names) in zip(out, fields.values()):
        codes = re.findall("[a-zA-Z]", block.format)
        assert len(codes) == len(names)
        want = []
        for i, c in enumerate(codes):
            before = "".join(codes[:i])
            want.append(struct.calcsize(before + c) - struct.calcsize(c))
        assert [int(v) for v in line.split()] == want + [block.size]


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
