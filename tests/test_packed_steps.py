"""The order of waits of the packed state kernel's data warps (csrc/steps_done.h), over every interleaving
of a model of its warps (no GPU needed)."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "linear_attention_sequence_chunkwise_b200", "csrc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("model") / "packed_steps")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, os.path.join(HERE, "packed_steps_model.cpp"), "-o", out], check=True)

    def run(rule, chunks):
        return subprocess.run([out, str(rule), *map(str, chunks)], check=True, capture_output=True, text=True,
                              timeout=60).stdout.strip()
    return run


# a chunk of 128 tokens has two steps; one of up to 64, a sequence's last, has one (dealt-out chunks: anywhere)
CHUNKS = [[1], [2], [2, 1], [2, 2], [2, 2, 2, 1], [1, 1, 1], [1, 2, 1, 2], [2, 2, 2, 2, 2], [1, 2, 2, 1, 1, 2]]


@pytest.mark.parametrize("chunks", CHUNKS)
def test_waits_always_end(model, chunks):
    assert model(1, chunks) == "ok"


@pytest.mark.parametrize("chunks", [[2, 2], [2, 2, 2, 1], [1, 2, 1, 2]])
def test_a_second_wait_for_a_step_may_not_end(model, chunks):
    """What the rule is for: where a step is waited for twice, an interleaving leaves a warp waiting."""
    assert model(0, chunks) == "stuck"
