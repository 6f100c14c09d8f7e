"""What the compiler made of the key/value cache's kernels, read from the assembly
of code built here (CPU only: hipcc cross-compiles)."""
import os
import re
import shutil

import pytest

pytest.importorskip("torch")

from hadamard_rotated_w4a4_amd import build as hip  # noqa: E402
from test_kernel_code import assembly, instructions, kernels, waits_between  # noqa: E402

pytestmark = pytest.mark.skipif(shutil.which(hip.HIPCC) is None, reason=f"no compiler at {hip.HIPCC}")


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    return assembly(os.path.join(hip.CSRC, "kv.hip"), tmp_path_factory.mktemp("code") / "kv.s")


def test_no_kernel_spills(code):
    """Nothing in scratch memory: its loads would share a counter with the direct
    loads to LDS, and a spilt sum would cost more than the products."""
    parts = code.split("  - .agpr_count:")[1:]
    names = [re.search(r"\.name: +(\S+)", p).group(1) for p in parts]
    assert len([n for n in names if "attend_tile_kernel" in n]) == 18 and len([n for n in names if "attend_stream_kernel" in n]) == 12
    for name, part in zip(names, parts):
        for what in ("private_segment_fixed_size", "vgpr_spill_count"):
            assert int(re.search(rf"\.{what}: +(\d+)", part).group(1)) == 0, (name, what)


def test_direct_loads_wait_for_their_m0(code):
    for name in kernels(code, "attend_tile_kernel"):
        lines = instructions(code, name)
        loads = [i for i, (line, _) in enumerate(lines) if "load_lds" in line]
        assert loads, name
        for i in loads:
            write = max(j for j, (line, _) in enumerate(lines[:i]) if re.match(r"s_\w+ m0,", line))
            assert waits_between(lines, write, i) >= 1, (name, lines[write:i + 1])


def test_the_loop_keeps_its_sums_and_its_loads(code):
    """Between the first and the last product of a tile's loop: sums stay where they
    are, and no wait is for the direct loads, which the compiler does not count."""
    for name in kernels(code, "attend_tile_kernel"):
        lines = [line for line, inline in instructions(code, name) if not inline]
        products = [i for i, line in enumerate(lines) if "v_mfma" in line]
        # the two runs of products, whichever the compiler put first
        cut = max(range(1, len(products)), key=lambda i: products[i] - products[i - 1])
        for run in (products[:cut], products[cut:]):
            body = lines[run[0]:run[-1] + 1]
            assert sum(line.startswith(("v_mov_b32", "v_accvgpr")) for line in body) <= 4, name
            assert not [line for line in body if "vmcnt" in line], name
