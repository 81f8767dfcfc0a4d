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


@pytest.mark.parametrize("block", [0, 100000])
def test_a_window_without_order_is_planned_by_all_the_keys_its_rows_see(block):
    """A window limits how far back a query looks. Where no order (or a long block) lets it look
    ahead to the chunk's end, 4,096 queries on an empty cache walk up to 4,096 keys each, with a
    window of 16 as without one, and few workgroups have to share them."""
    from bidirectional_mamba_state_amd import bdssm
    d = bdssm.attn_dims(1, 1, 1, 64, bdssm.BF16, 64)
    whole = bdssm.attn_step_workspace(d, 4096, 0, bdssm.attn_mask(0.125, block))
    windowed = bdssm.attn_step_workspace(d, 4096, 0, bdssm.attn_mask(0.125, block, 16))
    assert whole == windowed > 0
    assert bdssm.attn_step_workspace(d, 4096, 0, bdssm.attn_mask(0.125, 1, 16)) == 0  # 16 keys back, none ahead
