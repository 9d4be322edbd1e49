"""Exhaustive CPU check of the quotient the int8 row quantisation uses
(quotient_i8_check.c): its code is the IEEE division's for every pair of bf16
numbers up to the largest. The range in which the kernels take the two-float
quotient is read from their source."""

import os
import re
import shutil
import subprocess

import numpy as np
import pytest

from memory_bound_w8a8_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "quotient_i8_check.c")

pytestmark = pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")


def _run(tmp_path, *defines):
    exe = str(tmp_path / "i8")
    subprocess.run(["gcc", "-O2", "-fopenmp", "-ffp-contract=off", *[f"-D{d}" for d in defines], SRC, "-lm", "-o", exe],
                   check=True)
    env = dict(os.environ, OMP_NUM_THREADS=str(min(16, os.cpu_count() or 1)))
    proc = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True, env=env, timeout=600)
    fields = proc.stdout.split()
    return proc.returncode, {fields[i]: int(fields[i + 1]) for i in range(0, len(fields), 2)}, proc.stderr


def test_code_is_the_divisions_for_every_bf16_pair(tmp_path):
    rc, stats, err = _run(tmp_path)
    p = np.arange(31 << 7, 0x7F7F + 1, dtype=np.int64)
    assert stats["pairs"] == 2 * int(np.sum(p + 1))
    assert 0 < stats["two_floats"] < stats["pairs"]
    assert stats["differ"] == 0 and rc == 0, err[:2000]


def test_two_floats_alone_miss_codes_of_the_largest_rows(tmp_path):
    rc, stats, err = _run(tmp_path, "NO_TOP")
    assert rc == 1 and stats["differ"] == 10  # five pairs, both signs
    assert all(float.fromhex(line.split()[1]) >= 2.0 ** 125 for line in err.splitlines())


def test_kernels_take_the_two_floats_in_the_checked_range():
    source = open(os.path.join(build.CSRC, "norm_quant.hip")).read()
    body = source[source.index("v2u codes8_i8("):]
    body = body[:body.index("\n}\n")]
    assert re.search(r"if \(amax >= 0x1p-96f && amax < 0x1p100f\)", body)
