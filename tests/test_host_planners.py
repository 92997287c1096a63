"""The host planners of the attention calls under AddressSanitizer and UndefinedBehaviorSanitizer, on
the CPU: planner_checks.hip includes their sources and checks tables, parts, shares and overlaps of
random batches.  (Only the host pass is instrumented; no kernel is launched.)"""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def test_planners_cover_every_step_once(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is not available")
    from pool_score_top_amd import build as B
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC", "-O3")] + ["-O1", "-Wno-unused-function"]
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host",
           "-fno-sanitize-recover=undefined"]
    csrc = os.path.join(ROOT, "pool_score_top_amd", "csrc")
    exe, objs, procs = str(tmp_path / "planner_checks"), [], []
    # (layer.hip is part of the checks' own unit)
    for src, extra in [(os.path.join(ROOT, "tests", "planner_checks.hip"), san)] + [
            (os.path.join(csrc, s), B.FILE_FLAGS.get(s, []))
            for s in B.SOURCES if s not in ("layer.hip", "attend.hip", "attend_bwd.hip")]:
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        procs.append(subprocess.Popen([HIPCC, *flags, *extra, "-c", src, "-o", objs[-1]],
                                      stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    for p in procs:
        out, _ = p.communicate()
        assert p.returncode == 0, out[-4000:]
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address", "-Xarch_host",
                        "-fsanitize=undefined", "-o", exe, *objs], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe, "2000"], capture_output=True, text=True, timeout=600,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert r.stdout.startswith("ok: 2000 batches")
    assert int(r.stdout.split(",")[1].split()[0]) > 100
