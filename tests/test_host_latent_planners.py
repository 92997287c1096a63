"""The shares of the latent attention on the CPU: of the absorbed form, which every workgroup finds for
itself (latent_planner_checks.hip), and of the expanded form's backward pass, whose units count more than
their steps (the checks of planner_checks.hip with the expanded form's costs).  (Only the host pass is
instrumented; no kernel is launched.)"""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]


def run(tmp_path, sources, count):
    from pool_score_top_amd import build as B
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC", "-O3")] + ["-O1", "-Wno-unused-function"]
    objs, procs = [], []
    for src, extra in sources:
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        procs.append(subprocess.Popen([HIPCC, *flags, *extra, "-c", src, "-o", objs[-1]],
                                      stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    for p in procs:
        out, _ = p.communicate()
        assert p.returncode == 0, out[-4000:]
    exe = str(tmp_path / "checks")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN, "-o", exe, *objs], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe, str(count)], capture_output=True, text=True, timeout=600,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0 and r.stdout.startswith(f"ok: {count} batches"), (r.stdout + r.stderr)[-4000:]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is not available")
def test_every_tile_is_in_one_share(tmp_path):
    from pool_score_top_amd import build as B
    stop = ["-Xarch_host", "-fno-sanitize-recover=undefined"]
    run(tmp_path, [(os.path.join(ROOT, "tests", "latent_planner_checks.hip"), SAN + stop + B.FILE_FLAGS["latent.hip"])],
        2000)


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is not available")
def test_every_step_of_the_expanded_backward_is_in_one_share(tmp_path):
    from pool_score_top_amd import build as B
    stop = ["-Xarch_host", "-fno-sanitize-recover=undefined"]
    csrc = os.path.join(ROOT, "pool_score_top_amd", "csrc")
    text = open(os.path.join(ROOT, "tests", "planner_checks.hip")).read()
    for a, b in (("plan_attend_bwd(cq, ck, b.nseq, b.Hq, b.Hkv)", "plan_attend_bwd(cq, ck, b.nseq, b.Hq, b.Hkv, true)"),
                 ("x.second.n0, b.G).steps", "x.second.n0, b.G, true).steps"),
                 ("return keys_cost(lk, lq, n0, b.G);", "return keys_cost(lk, lq, n0, b.G, true);"),
                 ('#include "../pool_score_top_amd/csrc/', f'#include "{csrc}/')):
        assert a in text
        text = text.replace(a, b)
    own = tmp_path / "expanded_checks.hip"
    own.write_text(text)
    run(tmp_path, [(str(own), SAN + stop + [f"-I{ROOT}/tests"])] + [
        (os.path.join(csrc, s), B.FILE_FLAGS.get(s, [])) for s in B.SOURCES
        if s not in ("layer.hip", "attend.hip", "attend_bwd.hip")], 2000)
