"""The tests' copy of the 4-bit products' launch rules has the sources' constants (CPU)."""
import os
import re

import _w4_rules as rules
from fp8_block_scaled_04_amd import build


def test_constants_are_those_of_the_sources():
    launch = open(build.W4_SOURCE).read()
    kernel = open(os.path.join(build.CSRC, "w4_kernel.hpp")).read()
    value = lambda text, name: eval(re.search(rf"\b{name} = ([0-9 *]+)", text).group(1))
    assert (rules.SPLIT8, rules.SPLIT4, rules.STREAM_SETS, rules.STREAM_BYTES, rules.STREAM_WORKGROUPS) == tuple(
        value(launch, n) for n in ("kSplit8", "kSplit4", "kStreamSets", "kStreamBytes", "kStreamWorkgroups"))
    assert (rules.WAVES, rules.LDS_BYTES) == (value(kernel, "kW4Waves"), value(kernel, "kW4LdsBytes"))
    assert "kBlocks = deep(5)" in kernel and f"kBlocks = {rules.STREAM_DEPTH};" in kernel


def test_copy_of_the_rules():
    """Shapes whose kernels a profile named: tile, rows, steps and whether whole rows a wave."""
    for args, want in [((1, 4096, 7168, 128, False), (1, 1, 2, False)), ((5, 2111, 7168, 32, False), (8, 1, 2, False)),
                       ((16, 7168, 16384, 128, True), (16, 2, 1, False)), ((8, 4096, 2048, 64, True, 64), (1, 1, 2, True)),
                       ((512, 7168, 2048, 128, False, 128), (16, 2, 1, True))]:
        p = rules.plan(*args)
        assert (p.tokens, p.rows, p.steps, p.streamed) == want
