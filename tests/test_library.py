"""The two links of the library: libmuon.so needs nothing but the NVIDIA driver
of the machine it is loaded on, and has every entry point; the Python face's
shares the process's CUDA runtime."""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def libs():
    from newton_schulz_06_gb300 import build as b
    b.build()
    return b.LIB, b.TORCH_LIB


def needed(path):
    out = subprocess.run(["readelf", "-d", path], capture_output=True, text=True, check=True).stdout
    return re.findall(r"\(NEEDED\).*\[(.*)\]", out)


def test_the_c_library_needs_no_cuda_library(libs):
    assert not [n for n in needed(libs[0]) if "cuda" in n or "cudart" in n]
    assert any(n.startswith("libcudart") for n in needed(libs[1]))


def test_both_have_every_entry_point(libs):
    from newton_schulz_06_gb300 import _lib
    for path in libs:
        out = subprocess.run(["nm", "-D", "--defined-only", path], capture_output=True, text=True,
                             check=True).stdout
        syms = set(re.findall(r"\bT (\w+)", out))
        assert syms == set(_lib.EXPORTS)


def test_the_c_library_loads_without_a_toolkit(libs, tmp_path):
    """In a process that has no CUDA library and cannot find one, the library
    loads and answers: here with the refusal of a call without arguments."""
    code = (
        "import ctypes, sys\n"
        "L = ctypes.CDLL(sys.argv[1])\n"
        "buf = ctypes.create_string_buffer(64)\n"
        "assert L.muon_layer_norm(None, None, buf, 64) == -1 and buf.value == b'args is NULL'\n"
        "assert 'libcudart' not in open('/proc/self/maps').read()\n")
    copy = tmp_path / "libmuon.so"
    copy.write_bytes(open(libs[0], "rb").read())
    env = {k: v for k, v in os.environ.items() if k not in ("LD_LIBRARY_PATH", "LD_PRELOAD")}
    subprocess.run([sys.executable, "-c", code, str(copy)], check=True, env=env, cwd=tmp_path, timeout=120)
