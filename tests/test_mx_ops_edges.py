"""CPU tests of corners of the operators around the MX products."""
import os
import re

import dense_gemm_epilogue_tiled_amd as gr

CSRC = os.path.join(os.path.dirname(gr.__file__), "csrc")


def test_flag_of_unusual_scales_is_written_by_its_wave_alone():
    """No barrier orders a workgroup's start and its first turn, so a word that one thread clears and any wave sets
    can lose a wave's 1. Each wave writes a word of its own, whatever its value, before the turn's barrier, and
    nothing else writes there: the words hold the waves' flags after the last barrier in any order of the waves."""
    text = open(os.path.join(CSRC, "w4_stream.hpp")).read()
    assert "int again[NW]" in text
    writes = re.findall(r"lds\.again(\[[^\]]*\])?\s*=[^=]\s*([^;]*);", text)
    assert writes == [("[wave]", "bad")]
    at = text.index("lds.again[wave] = bad")
    assert re.match(r"[^;]*;\s*\}?\s*lds_barrier\(\);", text[at:])
