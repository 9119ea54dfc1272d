"""The weight gradient's waits, played through on the CPU with loads that land
in any order (weight_grad_stages.cpp, which includes the header that the
kernel takes its stages and phases from)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("stages") / "model")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I",
                    os.path.join(ROOT, "newton_schulz_06_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "weight_grad_stages.cpp"), "-o", exe], check=True)

    def run(guard):
        out = subprocess.run([exe, str(guard)], capture_output=True, text=True, check=True).stdout
        return [int(v) for v in out.split()]
    return run


def test_no_step_takes_another_steps_stage(model):
    assert model(1) == [0, 0]


def test_the_model_finds_the_missing_wait(model):
    """Without the wait for a stage's last user, a slow load is enough to go
    wrong in either shape."""
    narrow, wide = model(0)
    assert narrow > 0 and wide > 0


def test_the_kernel_waits_for_the_stages_last_user():
    """The one place where a step's decoding begins has the wait, for both
    shapes."""
    text = open(os.path.join(ROOT, "newton_schulz_06_gb300", "csrc", "weight_grad.cu")).read()
    wait = text[text.index("const uint32_t last = last_user<WIDE>(step);"):]
    wait = wait[:wait.index("uint4 q[")]
    assert "if constexpr" not in wait and "stage_was_used<WIDE>(step)" in wait
    assert "WIDE ? there() && used() : used() && there()" in wait
