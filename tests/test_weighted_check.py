"""The dispatch kernel's quotient of weighted rows against the oracle's IEEE
quotient (CPU only; see weighted_check.c)."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("wc") / "weighted_check")
    cmd = ["gcc", "-O2", "-std=c11", "-ffp-contract=off", "-fno-fast-math", "-fopenmp",
           os.path.join(HERE, "weighted_check.c"), os.path.join(ROOT, "oracle", "bfp8_oracle.c"), "-lm", "-o", exe]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    return exe


def _run(exe, groups):
    out = subprocess.run([exe, str(groups)], check=True, capture_output=True, text=True).stdout
    return [int(kv.split("=")[1]) for kv in out.split()]


def test_weighted_quotient(program):
    tot, bad, one = _run(program, 5000)
    assert tot == 5000 * 0x401 * 2 and bad == 0
    assert one > tot // 10000      # the check reaches the ties that a single product misses


@pytest.mark.slow
def test_weighted_quotient_of_many_groups(program):
    tot, bad, _ = _run(program, 500_000)
    assert tot > 1_000_000_000 and bad == 0
