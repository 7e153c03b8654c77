"""The planner of attention with sinks and over a shared prefix, under
sanitizers."""

import os

from test_host_sanitizers import CSRC, HOST, ROOT, SAN, _build_and_run


def test_shared_planner_under_asan_ubsan(tmp_path):
    out = _build_and_run(
        ["g++", "-std=c++17"] + SAN + ["-I", os.path.join(ROOT, "include"), "-I", CSRC,
                                       os.path.join(CSRC, "plan.cpp"), os.path.join(CSRC, "kv_plan.cpp"),
                                       os.path.join(HOST, "sanitize_kv_shared.cpp")],
        str(tmp_path / "sanitize_kv_shared"), "shared planner sweep done")
    assert int(out.split("(")[1].split()[0]) > 10000, out
