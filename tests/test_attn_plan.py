"""Launch plans of the paged-cache attention and its workspace query, on the CPU
(tests/attn_plan_check.cc linked against the library's objects)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "bidirectional_mamba_state_amd")


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not installed")
def test_a_workspace_serves_every_shorter_cache(tmp_path):
    from bidirectional_mamba_state_amd import build
    objs = [os.path.join(PACKAGE, "_build", os.path.splitext(s)[0] + ".o") for s in build.SOURCES]
    if not all(os.path.exists(o) for o in objs):
        build.build()
    exe = str(tmp_path / "attn_plan_check")
    cmd = ["hipcc", "--offload-arch=gfx950", "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(PACKAGE, "csrc"), "-x", "hip", os.path.join(ROOT, "tests", "attn_plan_check.cc"),
           "-x", "none", *objs, "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout
