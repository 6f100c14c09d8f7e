"""What the compiler made of the kernels' inline assembly, read from the assembly
of code built here (CPU only: hipcc cross-compiles)."""
import os
import re
import shutil
import subprocess

import pytest

pytest.importorskip("torch")

from hadamard_rotated_w4a4_amd import build as hip  # noqa: E402

pytestmark = pytest.mark.skipif(shutil.which(hip.HIPCC) is None, reason=f"no compiler at {hip.HIPCC}")


def assembly(source, out):
    """Device assembly of a .hip file, with the library's own flags."""
    flags = [f for f in hip.FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([hip.HIPCC, *flags, "-I", os.path.join(hip.ROOT, "include"), "-I", hip.CSRC, "--cuda-device-only", "-S",
                    "-o", str(out), str(source)], check=True, capture_output=True, text=True)
    return open(out).read()


def instructions(text, kernel):
    """(instruction lines of a kernel, whether each came from inline assembly)."""
    body = text[text.index(f"\n{kernel}:"):]
    body = body[:body.index("s_endpgm")]
    lines, inline = [], False
    for line in body.splitlines():
        if "#ASMSTART" in line or "#ASMEND" in line:
            inline = "#ASMSTART" in line
            continue
        line = line.split(";")[0].strip()
        if line and not line.startswith(".") and not line.endswith(":"):
            lines.append((line, inline))
    return lines


def waits_between(code, i, j):
    """Wait states between instructions i and j: one an instruction, n + 1 an s_nop n."""
    return sum(int(line.split()[1]) + 1 if line.startswith("s_nop") else 1 for line, _ in code[i + 1:j])


PROBE = """
#include "common.h"
#include "{header}"
using namespace w4a4;
typedef const __attribute__((address_space(1))) void global;
typedef __attribute__((address_space(3))) void shared;
extern "C" __global__ void probe(const uint8_t *p, uint8_t *y, int on) {{
    __shared__ uint8_t smem[4096];
    const uint32_t base = (uint32_t)(uintptr_t)(shared *)smem;
    __builtin_amdgcn_global_load_lds((global *)(p + 4 * threadIdx.x), (shared *)(smem + 1024), 4, 0, 0);
    {load};
    __builtin_amdgcn_global_load_lds((global *)(p + 256 + 4 * threadIdx.x), (shared *)(smem + 1024), 4, 0, 0);
    __builtin_amdgcn_s_waitcnt(0);
    y[threadIdx.x] = smem[threadIdx.x] + smem[1024 + threadIdx.x];
}}
"""


@pytest.mark.parametrize("header,load", [("k_mx4.h", "mx4_load16(p + 16 * threadIdx.x, base)"),
                                         ("k_mx4.h", "mx4_load16(p + 16 * threadIdx.x, base, on)"),
                                         ("k_dense.h", "dma16s(p, 16 * threadIdx.x, base)")])
def test_direct_loads_say_that_they_write_m0(tmp_path, header, load):
    """Between two of the compiler's own direct loads to one LDS address, one of
    ours to another: the compiler must set M0 again after it, and ours needs a
    wait state between its write of M0 and its load."""
    source = tmp_path / "probe.hip"
    source.write_text(PROBE.format(header=header, load=load))
    code = instructions(assembly(source, tmp_path / "probe.s"), "probe")
    ours = [i for i, (line, inline) in enumerate(code) if inline and "load_lds" in line]
    later = [i for i, (line, inline) in enumerate(code) if not inline and "load_lds" in line and i > ours[-1]]
    assert len(ours) == 1 and len(later) == 1
    write = max(i for i, (line, _) in enumerate(code[:ours[0]]) if line.startswith("s_mov_b32 m0,"))
    assert code[write][1] and waits_between(code, write, ours[0]) >= 1
    between = [line for line, inline in code[ours[0] + 1:later[0]] if not inline]
    assert any(re.match(r"s_\w+ m0,", line) for line in between), between


@pytest.fixture(scope="module")
def product(tmp_path_factory):
    """Assembly of the MXFP4 product's kernels."""
    return assembly(os.path.join(hip.CSRC, "mx4.hip"), tmp_path_factory.mktemp("code") / "mx4.s")


def kernels(text, name):
    return sorted(set(re.findall(rf"^(_ZN4w4a4\d+{name}\w*):", text, re.M)))


def test_streams_wait_for_their_rows_by_a_load_that_follows_them(product):
    """A stream's first barrier needs the rows' codes in LDS, direct loads that the
    compiler does not count.  It waits for the scales, loaded after the codes
    (loads return in order): by waits of the compiler's own, which count what it
    issued behind them, and by no count of ours."""
    names = kernels(product, "gemm_mx4_stream_kernel")
    assert len(names) == 5
    for name in names:
        code = instructions(product, name)
        assert not [line for line, inline in code if inline and "s_waitcnt" in line], name
        first = next(i for i, (line, _) in enumerate(code) if line == "s_barrier")
        direct = max(i for i, (line, _) in enumerate(code[:first]) if "load_lds" in line)
        behind = [line for line, _ in code[direct + 1:first] if re.match(r"(global|buffer|flat)_(load|store)", line)]
        waits = [int(re.search(r"vmcnt\((\d+)\)", line).group(1)) for line, _ in code[direct + 1:first] if "vmcnt" in line]
        assert waits and min(waits) < len(behind), f"{name}: {len(behind)} loads behind the codes, waits {waits}"


def test_the_plan_counts_the_workgroups_that_a_cu_holds(product):
    """kShapes' workgroups per CU against the kernels' LDS and registers (160 KB of
    LDS; 512 VGPRs a SIMD in groups of 8 to at most 8 waves, four SIMDs)."""
    host = open(os.path.join(hip.CSRC, "mx4.hip")).read()
    configs = dict(re.findall(r"using (T\w+) = Mx4Cfg<([\d, ]+)>;", host))
    per_cu = dict(re.findall(r"shape<(T\w+)>\((\d+),", host))
    assert len(configs) == 6 and per_cu.keys() == configs.keys()
    for shape, args in configs.items():
        numbers = [int(n) for n in args.split(",")]
        kernel = "gemm_mx4_tile_kernelINS_6Mx4CfgI" + "".join(f"Li{n}E" for n in numbers) + "EE"
        meta = next(part for part in product.split("  - .agpr_count:")[1:] if kernel in part)
        lds, vgprs, scratch = (int(re.search(rf"\.{name}: +(\d+)", meta).group(1)) for name in
                               ("group_segment_fixed_size", "vgpr_count", "private_segment_fixed_size"))
        waves = numbers[0] * numbers[1]
        slots = min(8, 512 // ((vgprs + 7) // 8 * 8)) * 4
        assert scratch == 0 and min(160 * 1024 // lds, slots // waves) == int(per_cu[shape]), (shape, lds, vgprs, waves)


def test_every_direct_load_waits_for_its_m0(product):
    """One wait state between a write of M0 and the load that reads it."""
    for name in kernels(product, "gemm_mx4_stream_kernel") + kernels(product, "gemm_mx4_tile_kernel"):
        code = instructions(product, name)
        loads = [i for i, (line, _) in enumerate(code) if "load_lds" in line]
        assert loads, name
        for i in loads:
            write = max(j for j, (line, _) in enumerate(code[:i]) if re.match(r"s_\w+ m0,", line))
            assert waits_between(code, write, i) >= 1, (name, code[write:i + 1])
