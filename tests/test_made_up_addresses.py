"""Tests that are not marked `gpu` hand made-up addresses to the library. Where
such a call passes every host check it ends in the device check without a GPU,
and would start a kernel on memory that nobody owns with one: those tests must
not run where a GPU is (CPU only)."""

import os
import subprocess
import sys

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
FILES = ["test_abi.py", "test_step_abi.py", "test_step_limits.py"]


def _session(word, *args, **env):
    proc = subprocess.run([sys.executable, "-m", "pytest", "-q", "-s", "-p", "device_reach", "-m", "not gpu", *args,
                           *(os.path.join(HERE, f) for f in FILES)], cwd=os.path.dirname(HERE), text=True,
                          env=dict(os.environ, PYTHONPATH=HERE, **env), stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    assert proc.returncode == 0, proc.stdout[-3000:]
    return {line.split(" ", 1)[1] for line in proc.stdout.splitlines() if line.startswith(word)}


@pytest.mark.skipif(torch.cuda.is_available(), reason="runs such calls: only without a GPU")
def test_calls_that_pass_the_host_checks_stay_away_from_gpus():
    reached = _session("REACHED ")
    assert any("test_device_error_without_gpu" in name for name in reached)  # the watch sees such calls
    without = _session("WITHOUT ", "--collect-only", DEVICE_REACH="gpu")
    assert reached <= without, f"would launch on made-up addresses: {sorted(reached - without)}"
