"""Calls of the latent attention on the CPU, under the sanitizers: latent_call_checks.hip.  (Only the host pass is
instrumented; no kernel is launched.)"""
import os

import pytest

from test_host_latent_planners import HIPCC, ROOT, SAN, run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is not available")
def test_keys_of_every_share_are_walked_once(tmp_path):
    """Lengths up to 2^31 - 256 among them, whose last block ends past 2^31."""
    from pool_score_top_amd import build as B
    stop = ["-Xarch_host", "-fno-sanitize-recover=undefined"]
    run(tmp_path, [(os.path.join(ROOT, "tests", "latent_call_checks.hip"), SAN + stop + B.FILE_FLAGS["latent.hip"])],
        2000)
