"""Calls of the latent attention on the CPU: under the sanitizers, latent_call_checks.hip (only the host pass is
instrumented; no kernel is launched), and what the workspace queries say against what the calls take."""
import os

import numpy as np
import pytest

from pool_score_top_amd import kpool as K
from test_gpu_latent import AT, _call
from test_host_latent_planners import HIPCC, ROOT, SAN, run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is not available")
def test_keys_of_every_share_are_walked_once(tmp_path):
    """Lengths up to 2^31 - 256 among them, whose last block ends past 2^31; parts within the workspace."""
    from pool_score_top_amd import build as B
    stop = ["-Xarch_host", "-fno-sanitize-recover=undefined"]
    run(tmp_path, [(os.path.join(ROOT, "tests", "latent_call_checks.hip"), SAN + stop + B.FILE_FLAGS["latent.hip"])],
        2000)


def _needs(nb, selected, **kw):
    """Whether a call of these sizes asks for more than nb bytes of workspace.  (Its output lies over its queries, which
    is refused behind that: nothing is launched.)"""
    rc = _call(selected, nb=nb, o=AT["q"], **kw)
    text = K.lib().kpool_last_error()
    assert (rc == K.KPOOL_EWORKSPACE and b"bytes of workspace" in text) or (rc == K.KPOOL_EINVAL and b"overlaps" in text)
    return rc == K.KPOOL_EWORKSPACE


def _takes_what_it_says(q_lens, H, R, P, max_len, width):
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    for selected, nb, kw in (
            (False, K.attend_latent_workspace_bytes(cu, max_len, H, R, P), dict(max_len=max_len)),
            (True, K.attend_latent_selected_workspace_bytes(int(cu[-1]), width, H, R, P), dict(width=width))):
        assert not _needs(nb, selected, cu=cu, H=H, R=R, P=P, **kw)
        assert nb == 0 or _needs(nb - 1, selected, cu=cu, H=H, R=R, P=P, **kw)


@pytest.mark.parametrize("q_lens,H,R,P", [
    ([5, 1, 1, 1, 1], 16, 64, 8), ([5] + [1] * 8, 8, 64, 8), ([33] + [1] * 600, 1, 64, 8), ([1024], 16, 512, 64),
    ([2] * 300, 16, 512, 64), ([2], 4, 64, 8)])
def test_lists_without_entries_take_the_workspace_they_ask_for(q_lens, H, R, P):
    _takes_what_it_says(q_lens, H, R, P, 0, 0)


def test_calls_take_the_workspace_they_ask_for():
    g = np.random.default_rng(3)
    for _ in range(300):
        q_lens = g.integers(0, 4, g.integers(1, 60)) if g.random() < 0.7 else g.integers(0, 300, g.integers(1, 6))
        if q_lens.sum() == 0:
            q_lens[0] = 1
        _takes_what_it_says(q_lens, int(g.integers(1, 140)), 8 * int(g.integers(1, 65)), 8 * int(g.integers(0, 9)),
                            int(g.integers(0, 30000)), int(g.integers(0, 3000)) * int(g.integers(0, 2)))


@pytest.mark.parametrize("far", [2 ** 32 + 64, 2 ** 31, -2 ** 31 - 1, 2 ** 40])
def test_numbers_past_32_bits_are_refused(far):
    """ctypes passes the low 32 bits of a number: 2^32 + 64 would be 64."""
    import torch
    sizes = dict(max_len=640, H=16, R=512, P=64)
    for name in sizes:
        with pytest.raises(ValueError, match="32 bits"):
            K.attend_latent_workspace_bytes([0, 1], **{**sizes, name: far})
    sizes = dict(Tq=5, width=64, H=16, R=512, P=64)
    for name in sizes:
        with pytest.raises(ValueError, match="32 bits"):
            K.attend_latent_selected_workspace_bytes(**{**sizes, name: far})
    sizes = dict(Hq=16, Hkv=16, D=128, P=64)
    for fn in (K.attend_expanded_workspace_bytes, K.attend_expanded_backward_workspace_bytes):
        for name in sizes:
            with pytest.raises(ValueError, match="32 bits"):
                fn([0, 5], [0, 5], **{**sizes, name: far})
    q, cu = torch.zeros(1, 2, 16), np.array([0, 1], dtype=np.int32)
    with pytest.raises(ValueError, match="32 bits"):
        K.attend_latent(q, torch.zeros(4, 16), 8, cu, torch.from_numpy(cu), torch.ones(1), far, 0.1)
    for fn in (K.rotary, K.rotary_backward):
        with pytest.raises(ValueError, match="32 bits"):
            fn(q, torch.zeros(1), torch.zeros(4), begin=far)
