"""The rotary, scored-attention and page entry points' host code under AddressSanitizer
and UndefinedBehaviorSanitizer, on the CPU: tests/sanitize/paged_layer_check.c linked against the
host code of rotary.hip, pages.hip, attn.hip and attn_mfma.hip built with the sanitizers on the host side
only (the other objects are the regular ones; nothing reaches a GPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bidirectional_mamba_state_amd", "csrc")
OBJ = os.path.join(ROOT, "bidirectional_mamba_state_amd", "_build")
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")


def _run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout}\n{r.stderr}"
    return r


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not installed")
def test_paged_layer_host_code_under_sanitizers(tmp_path):
    from bidirectional_mamba_state_amd import build
    checked = ("rotary", "pages", "attn", "attn_mfma")
    others = [os.path.join(OBJ, os.path.splitext(s)[0] + ".o") for s in build.SOURCES if os.path.splitext(s)[0] not in checked]
    if not all(os.path.exists(o) for o in others):
        build.build()
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]
    objs = []
    for src in checked:
        o = str(tmp_path / (src + ".o"))
        _run(["hipcc", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", *san,
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
              "-I", os.path.join(ROOT, "include"), "-c", "-o", o, os.path.join(CSRC, src + ".hip")])
        objs.append(o)
    exe = str(tmp_path / "paged_layer_check")
    _run(["hipcc", "--offload-arch=gfx950", "-O1", "-g", *san, "-I", os.path.join(ROOT, "include"), "-x", "c++",
          os.path.join(ROOT, "tests", "sanitize", "paged_layer_check.c"), "-x", "none", *objs, *others, "-o", exe])
    assert "ok" in _run([exe], env=ENV).stdout
