"""Host code of the library on a stand-in for the HIP runtime (fake_gpu.py):
what is launched, in what order, and what is refused."""

import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("fake") / "fake_hip.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fPIC", "-shared",
                    os.path.join(HERE, "host", "fake_hip.cpp"), "-o", out], check=True)
    return out


def run(stand_in, check):
    r = subprocess.run([sys.executable, os.path.join(HERE, "fake_gpu.py"), stand_in, check], capture_output=True,
                       text=True, timeout=200)
    assert r.returncode == 0 and r.stdout.strip().endswith("done"), (r.stdout + r.stderr)[-3000:]


def test_calls_are_whole(stand_in):
    run(stand_in, "calls_are_whole")


def test_plans_are_the_calls(stand_in):
    run(stand_in, "plans_are_the_calls")


def test_all_launches_or_none(stand_in):
    run(stand_in, "all_launches_or_none")


def test_no_exception_leaves(stand_in):
    run(stand_in, "no_exception_leaves")
