"""The layer norm's ring kernels when a bounded wait runs out: what a block
still has in flight, on the CPU, and the way to the caller, on the GPU."""
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "newton_schulz_06_gb300", "csrc")


def test_an_aborted_block_waits_for_what_it_asked_for(tmp_path):
    exe = str(tmp_path / "ring")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC,
                    os.path.join(ROOT, "tests", "norm_ring.cpp"), "-o", exe], check=True)
    assert subprocess.run([exe], capture_output=True, text=True, check=True).stdout.strip() == "0"


def test_no_copy_is_asked_for_after_a_wait_that_ran_out():
    """Behind the barrier that follows a ring's wait, the block leaves before
    it asks for a further row."""
    text = open(os.path.join(CSRC, "layer_norm.cu")).read()
    for name in ("norm_ring_kernel(const", "norm_grad_ring_kernel(const"):
        body = text[text.index(name):]
        body = body[body.index("ring_wait("):]
        assert body.index("if ((aborted = abort_flag") < body.index("load(r + ")


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported_once():
    import ctypes

    import newton_schulz_06_gb300 as ns
    from newton_schulz_06_gb300 import _lib
    buf = ctypes.create_string_buffer(128)
    stream = torch.cuda.current_stream().cuda_stream
    assert _lib.lib().muon_debug_ops_wait_timeout(0, stream, buf, 128) == _lib.MUON_ERR_INVALID_ARG
    ns.ops_sync()
    assert _lib.lib().muon_debug_ops_wait_timeout(100, stream, buf, 128) == 0
    with pytest.raises(ns.MuonError) as e:
        ns.ops_sync()
    assert e.value.code == _lib.MUON_ERR_TIMEOUT
    # the context is as usable as before, and the word has been cleared
    ns.ops_sync()
    x = torch.randn(3000, 7168, device="cuda").bfloat16()
    y, mean, rstd = ns.layer_norm(x)
    ns.layer_norm_backward(x, x, mean, rstd)
    ns.ops_sync()
