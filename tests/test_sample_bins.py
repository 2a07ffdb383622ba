"""The bins that the sampler's kernels index with, on the host, at the ends of temperatures and logits: a temperature of +inf
beside a logit of +inf once gave the largest logit the lowest bin, and distances that left the histograms."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("bins") / "sample_bins_check")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-fno-fast-math", os.path.join(HERE, "host", "sample_bins_check.cpp"), "-o", exe])
    return exe


def test_bins_stay_in_their_histograms(program):
    seen, bad = map(int, subprocess.check_output([program], text=True).split())
    assert seen > 10_000_000 and bad == 0, f"{bad} of {seen}"
