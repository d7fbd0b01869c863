"""The dispatch kernel's division-free quotient against the oracle's IEEE
quotient (CPU only; see reciprocal_check.c): a strided subset of the bf16 amax
values by default, all of them (about 1.07e9 (amax, x, sign) cases, each with
four reciprocal candidates) in the slow test."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("rc") / "reciprocal_check")
    cmd = ["gcc", "-O2", "-std=c11", "-ffp-contract=off", "-fno-fast-math", "-fopenmp",
           os.path.join(HERE, "reciprocal_check.c"), os.path.join(ROOT, "oracle", "bfp8_oracle.c"), "-lm", "-o", exe]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    return exe


def _run(exe, stride):
    out = subprocess.run([exe, str(stride)], check=True, capture_output=True, text=True).stdout
    fields = dict(kv.split("=") for kv in out.split())
    return int(fields["tot"]), int(fields["bad"])


def test_quotient_strided(program):
    tot, bad = _run(program, 97)
    assert tot > 5_000_000 and bad == 0


@pytest.mark.slow
def test_quotient_exhaustive(program):
    tot, bad = _run(program, 1)
    assert tot == 1_065_402_240 and bad == 0
