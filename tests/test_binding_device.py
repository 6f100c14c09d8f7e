"""The native binding leaves the caller's device current, also where a call raises
after it switched.  No GPU takes part: a stand-in for the four HIP calls on the
way there (two devices that only remember which is current), and a batched tensor
on the second one, which has no storage and whose data pointer cannot be had."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STAND_IN = """
static int current, switches;
int hipGetDeviceCount(int *n) { *n = 2; return 0; }
int hipGetDevice(int *d) { *d = current; return 0; }
int hipSetDevice(int d) { switches += d != current; current = d; return 0; }
int hipDeviceGetStreamPriorityRange(int *least, int *greatest) { *least = *greatest = 0; return 0; }
int stand_in_current(void) { return current; }
int stand_in_switches(void) { return switches; }
"""

CHILD = """
import ctypes, sys
hip = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # found ahead of the HIP runtime
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
torch.cuda.is_available = lambda: False  # a fake tensor would warm the device up
from hadamard_rotated_w4a4_amd import ops
ops._native()
with FakeTensorMode():
    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda:1")
    x, codes, scales = empty(2, 4, 64), empty(4, 32, dtype=torch.uint8), empty(4, 8, dtype=torch.uint8)
    start, before = hip.stand_in_current(), hip.stand_in_switches()
    try:
        torch.func.vmap(lambda one: ops.quantize_mx4(one, codes=codes, scales=scales))(x)
    except Exception as e:
        print("raised", type(e).__name__, str(e).splitlines()[0])
    print("switches", hip.stand_in_switches() - before, "start", start, "end", hip.stand_in_current())
"""


def test_a_call_that_raises_leaves_the_current_device(tmp_path):
    (tmp_path / "stand_in.c").write_text(STAND_IN)
    stand_in = str(tmp_path / "stand_in.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", stand_in, str(tmp_path / "stand_in.c")], check=True)
    out = subprocess.run([sys.executable, "-c", CHILD, stand_in], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert "raised" in out.stdout and "storage" in out.stdout, out.stdout + out.stderr
    assert "switches 2 start 0 end 0" in out.stdout, out.stdout + out.stderr
