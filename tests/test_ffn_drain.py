"""A CTA pair of the gated feed-forward kernels when a bounded wait runs out:
what it still has in flight, on the CPU (ffn_drain.cpp, which includes the
header that the kernel takes its rules from)."""
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "newton_schulz_06_gb300", "csrc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("drain") / "model")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, os.path.join(ROOT, "tests", "ffn_drain.cpp"), "-o", exe],
                   check=True)

    def run(rule):
        out = subprocess.run([exe, str(rule)], capture_output=True, text=True, check=True).stdout
        return [int(v) for v in out.split()]
    return run


def test_an_aborted_pair_waits_for_what_it_asked_for(model):
    assert model(1) == [0, 0]


def test_the_model_finds_loads_that_nobody_waits_for(model):
    """With each CTA's first thread waiting for the stages that it has loaded
    itself, pairs leave with loads in flight, and wait for bytes that nobody
    asked for."""
    left, stuck = model(0)
    assert left > 0 and stuck > 0


def test_the_pair_drains_after_all_roles_have_ended():
    """Behind the barrier at which both CTAs meet, whichever of them and
    whatever role gave up; and neither leaves before the other has drained."""
    text = open(os.path.join(CSRC, "gated_ffn.cu")).read()
    end = text[text.index("        if (OP == DHIDDEN) copies_done();"):]
    end = end[:end.index("tcgen05.dealloc")]
    assert end.index("cluster_sync_all()") < end.index("if (*abort_flag) give_up<OP>(") and end.count("return;") == 1
    last = text[text.index("void give_up("):]
    last = last[:last.index("\n}\n")]
    assert max(last.index("drain_loads<OP>("), last.index("commit_pair_local(")) < last.index("cluster_sync_all()")
    # whichever wait runs out, the other CTA learns of it before it meets this one
    body = text[text.index("bool wait_long("):]
    body = body[:body.index("\n}\n")]
    assert body.index("wait_bounded(") < body.index("store_cluster(")
    assert text.count("wait_bounded(") == 1 and text.count("wait_soon(") == 1       # that of the timeout test
    # each loading thread leaves its counts, whatever ended its loop
    body = text[text.index("load_operand(const FfnLaunch& p"):text.index("drain_loads(uint8_t*")]
    assert "return" not in body and body.index("= asked;") > body.rindex("load_box(")


def test_what_crosses_the_pair_is_released_to_it():
    """A barrier of the other CTA is arrived at by the tensor cores, by loads, or
    with the cluster's scope named; an arrival without one orders nothing
    beyond its own CTA."""
    text = open(os.path.join(CSRC, "gated_ffn.cu")).read() + open(os.path.join(CSRC, "tc_ptx.cuh")).read()
    arrivals = [line for line in text.splitlines() if "mbarrier.arrive" in line and "shared::cluster" in line
                and "tcgen05" not in line]
    assert arrivals and all(".cluster.shared::cluster" in line for line in arrivals)
    # the relaxed one only says that an accumulator has been read
    assert text.count("mbar_arrive_cluster_relaxed(tempty_leader") == 1


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported_once():
    import ctypes

    import newton_schulz_06_gb300 as ns
    from newton_schulz_06_gb300 import _lib
    buf = ctypes.create_string_buffer(128)
    stream = torch.cuda.current_stream().cuda_stream
    out_of_time = _lib.lib().muon_debug_ffn_wait_timeout
    assert out_of_time(0, stream, buf, 128) == _lib.MUON_ERR_INVALID_ARG
    ns.ops_sync()
    assert out_of_time(100, stream, buf, 128) == 0
    with pytest.raises(ns.MuonError) as e:
        ns.ops_sync()
    assert e.value.code == _lib.MUON_ERR_TIMEOUT
    # the context is as usable as before, and the word has been cleared
    ns.ops_sync()
    g = torch.Generator(device="cuda").manual_seed(1)
    x, *w = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((300, 64), (96, 64), (96, 64), (64, 96)))
    y, saved = ns.gated_ffn(x, *w)
    ns.gated_ffn_backward(y, x, saved, *w)
    ns.ops_sync()
