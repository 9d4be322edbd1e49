"""A pytest plugin (-p device_reach) for tests/test_made_up_addresses.py: tells
which tests call the library with arguments that pass all of its host checks
(without a GPU such a call ends in the device check), or, with
DEVICE_REACH=gpu, which tests would not run if a GPU were there."""

import os

import pytest
import torch

AS_WITH_GPU = os.environ.get("DEVICE_REACH") == "gpu"
FP8BQ_ERR_DEVICE = -4
_now = None
reached = set()

if AS_WITH_GPU:  # only to collect (--collect-only): nothing is run
    torch.cuda.is_available = lambda: True


class _Watched:
    """A function of the library that notes the running test where it ends in the device check."""

    def __init__(self, fn):
        object.__setattr__(self, "_fn", fn)

    def __call__(self, *args):
        out = self._fn(*args)
        if out == FP8BQ_ERR_DEVICE:
            reached.add(_now)
        return out

    def __setattr__(self, name, value):
        setattr(self._fn, name, value)

    def __getattr__(self, name):
        return getattr(self._fn, name)


def pytest_sessionstart(session):
    if AS_WITH_GPU:
        return
    import memory_bound_w8a8_amd as fp8bq
    from memory_bound_w8a8_amd import step

    library = step.step_lib()
    for name in (*fp8bq.EXPORTS, *fp8bq.STEP_EXPORTS):
        setattr(library, name, _Watched(getattr(library, name)))


@pytest.hookimpl(tryfirst=True)
def pytest_runtest_setup(item):
    global _now
    _now = item.nodeid


def pytest_collection_finish(session):
    if not AS_WITH_GPU:
        return
    for item in session.items:
        off = item.get_closest_marker("skip") or item.get_closest_marker("gpu") or any(
            bool(m.args and m.args[0]) for m in item.iter_markers("skipif"))
        if off:
            print(f"\nWITHOUT {item.nodeid}")


def pytest_sessionfinish(session):
    for name in sorted(reached):
        print(f"\nREACHED {name}")
