"""Calls from two host threads, on the CPU: the library's launches go to a fake
CUDA runtime (fake_cudart.c) that makes the threads' calls take a chosen
order."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import ctypes, sys, threading
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
from newton_schulz_06_gb300 import _lib
L = _lib.lib()
P = 1 << 20
which = sys.argv[3]


def call(cols):
    # many rows of bf16 on 16 bytes: the kernels that keep rows in a ring
    if which == "forward":
        a = _lib.LayerNormArgs(x=P, y=P, rows=20000, cols=cols, ld_x=cols, ld_y=cols, x_dtype=1, eps=1e-5)
        return L.muon_layer_norm(ctypes.byref(a), None, None, 0)
    a = _lib.LayerNormGradArgs(dy=P, x=2 * P, mean=P, rstd=P, dx=3 * P, rows=20000, cols=cols,
                               ld_dy=cols, ld_x=cols, ld_dx=cols, x_dtype=1)
    return L.muon_layer_norm_grad(ctypes.byref(a), None, 0, None, None, 0)


# two widths of one kernel, of which the second asks for less shared memory
# while the first is still between asking and launching
wide, narrow = int(sys.argv[4]), int(sys.argv[5])
fake.fake_hold()
got = {}
t = threading.Thread(target=lambda: got.setdefault("wide", call(wide)))
t.start()
while not fake.fake_held() and t.is_alive():
    pass
got["narrow"] = call(narrow)
t.join()
got["wide again"] = call(wide)
got["narrow again"] = call(narrow)
assert fake.fake_held()
print(sorted(got.items()), fake.fake_refused())
assert all(v == 0 for v in got.values()) and fake.fake_refused() == 0, got
"""


@pytest.mark.parametrize("which,wide,narrow", [("forward", 5120, 4800), ("backward", 4096, 2048)])
def test_two_threads_first_calls_of_one_kernel(tmp_path, which, wide, narrow):
    from newton_schulz_06_gb300 import build as b
    b.build()
    fake = str(tmp_path / "libfake.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-pthread", "-o", fake,
                    os.path.join(ROOT, "tests", "fake_cudart.c")], check=True)
    r = subprocess.run([sys.executable, "-c", CHILD, fake, ROOT, which, str(wide), str(narrow)],
                       env={**os.environ, "LD_PRELOAD": fake}, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
