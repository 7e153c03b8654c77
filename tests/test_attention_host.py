"""Host side of the attention operators: the planner under sanitizers, and
the diagnostic environment variables (read once per process, so each case
runs a child process)."""

import os
import subprocess
import sys

import pytest

import block_scaled_fp8_w8a16_amd as w8
from test_host_sanitizers import CSRC, HOST, ROOT, SAN, _build_and_run


def test_attention_planner_under_asan_ubsan(tmp_path):
    out = _build_and_run(
        ["g++", "-std=c++17"] + SAN + ["-I", os.path.join(ROOT, "include"), "-I", CSRC,
                                       os.path.join(CSRC, "plan.cpp"), os.path.join(CSRC, "kv_plan.cpp"),
                                       os.path.join(HOST, "sanitize_kv_plan.cpp")],
        str(tmp_path / "sanitize_kv_plan"), "attention planner sweep done")
    assert int(out.split("(")[1].split()[0]) > 100000, out


def child(code, **env):
    e = {k: v for k, v in os.environ.items() if k not in ("W8A16_LOG", "W8A16_DEBUG_SYNC")}
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=dict(e, **env),
                          capture_output=True, text=True, timeout=300)


BAD_SETTING = """
import block_scaled_fp8_w8a16_amd as w8
lib = w8.library()
print(lib.w8a16_rope_table(None, None, 1, 64, None))     # the setting is checked before the pointers
print(lib.w8a16_rope(*[0] * 17))
print(lib.w8a16_kv_append(None, None, None, None))
print(lib.w8a16_kv_attention(None, None, None, None))
print(repr(w8.last_error()))
print(w8.plan_kv_attention(1, 1, 100, 8, 1, 64).kernel)  # planning ignores it
"""


@pytest.mark.parametrize("var", ["W8A16_LOG", "W8A16_DEBUG_SYNC"])
def test_bad_setting_fails_every_call(var):
    r = child(BAD_SETTING, **{var: "yes"})
    assert r.returncode == 0, r.stderr[-3000:]
    lines = r.stdout.split("\n")
    assert lines[:4] == [str(w8.ERR_ENV)] * 4, r.stdout
    assert var in lines[4] and "must be 0 or 1" in lines[4]
    assert lines[5] == str(w8.KV_KERNEL_ROWS)


def test_launches_of_too_many_threads_are_refused():
    from test_attention import _descs
    from block_scaled_fp8_w8a16_amd.attention import RopeConfig
    lib = w8.library()
    assert lib.w8a16_rope_table(RopeConfig(1e4, 1, 0, 1, 4, 1, 0), 16, 1 << 26, 128, 0) == w8.ERR_SHAPE
    many = dict(s__seqs=1 << 22, s__tokens=1 << 22, s__max_new=1, c__kv_heads=8, ap__q_heads=8,
                at__q_heads=8, c__k_page_stride=1 << 20, c__v_page_stride=1 << 20,
                c__k_scale_page_stride=64, c__v_scale_page_stride=64)
    c, s, ap, at = _descs(**many)
    assert lib.w8a16_kv_append(c, s, ap, 0) == w8.ERR_SHAPE
    assert "too many" in w8.last_error()
    with pytest.raises(w8.W8A16Error) as e:
        w8.plan_kv_attention(1 << 22, 1, 64, 8, 8, 64)
    assert e.value.status == w8.ERR_SHAPE and "too many" in str(e.value)


LOGGED = """
import torch
import block_scaled_fp8_w8a16_amd as w8
cache = w8.kv_cache(8, 2, 32, 64)
table = w8.rope_table(256, 64)
bt = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
x = torch.randn(40, 2, 64, device="cuda").bfloat16()
q = torch.randn(40, 8, 64, device="cuda").bfloat16()
lens = torch.full((1,), 40, dtype=torch.int32, device="cuda")
w8.rope(x, table, torch.arange(40, dtype=torch.int32, device="cuda"))
for _ in range(2):      # each distinct launch is logged once
    q = w8.kv_append(cache, x, x, bt, lens, table=table, q=q)
    w8.kv_attention(q, cache, bt, lens)
    w8.kv_attention(q[:1], cache, bt, lens, plan_=w8.KVPlan(kernel=1, row_blocks=1, waves=4, chunk_tiles=1))
torch.cuda.synchronize()
"""


@pytest.mark.gpu
def test_log_of_the_attention_operators():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    r = child(LOGGED, W8A16_LOG="1", W8A16_DEBUG_SYNC="1")
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    log = [ln[7:] for ln in r.stderr.split("\n") if ln.startswith("w8a16: ")]
    assert len(log) == 5, log
    want = ["w8a16_rope_table positions=256 rot_dim=64", "w8a16_rope tokens=40 heads=2 head_dim=64",
            "w8a16_kv_append tokens=40 seqs=1 kv_heads=2", "w8a16_kv_attention tokens=40 seqs=1",
            "w8a16_kv_attention tokens=1 seqs=1"]
    for line, start in zip(log, want):
        assert line.startswith(start), line
    assert "kernel=kv-tile" in log[3] and "caller's plan" not in log[3]
    assert "kernel=kv-rows" in log[4] and log[4].endswith("caller's plan") and "chunks=4" in log[4]
