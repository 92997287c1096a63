"""kpool_attend_backward against the gradients' formulas in 64 bits (tolerances:
attend_reference.py) and against differences."""
import ctypes

import numpy as np
import pytest
import torch

from attend_reference import check_backward, cu_of, make
from pool_score_top_amd import kpool as K

BF16 = torch.bfloat16


def gradients(q_lens, k_lens, Hq, Hkv, D, seed, pad=0, gain=2.0):
    cu_q, cqd = cu_of(q_lens)
    cu_k, ckd = cu_of(k_lens)
    cu = (cu_q, cqd, cu_k, ckd)
    q, k, v = make(cu_q, cu_k, Hq, Hkv, D, seed, pad, gain)
    g = torch.Generator().manual_seed(seed + 1)
    d_o = torch.randn(int(cu_q[-1]), Hq, D, generator=g).to(BF16).cuda()
    o, lse = K.attend(q, k, v, *cu, want_lse=True)
    out = K.attend_backward(d_o, q, k, v, o, lse, *cu)
    check_backward(q, k, v, d_o, o, lse, cu_q, cu_k, 1.0 / D ** 0.5, *out)
    return q, k, v, d_o, o, lse, cu, out


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 8), (4, 4, 16), (4, 1, 64), (8, 2, 72), (6, 2, 128),
                                      (5, 1, 120), (40, 1, 64), (33, 1, 128)])
def test_packed_prompts(Hq, Hkv, D):
    lens = [1, 31, 0, 32, 33, 127, 128, 129, 300, 2]
    gradients(lens, lens, Hq, Hkv, D, Hq * 1000 + D)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 128), (12, 4, 64)])
def test_chunks_of_prompts(Hq, Hkv, D):
    """Queries at the end of longer keys; a sequence without queries, whose keys get 0."""
    *_, (dq, dk, dv) = gradients([5, 100, 0, 1, 260], [50, 1000, 77, 2000, 261], Hq, Hkv, D, Hq)
    assert (dk[1050:1127] == 0).all() and (dv[1050:1127] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 300])
def test_rows_without_keys(rows):
    *_, (dq, dk, dv) = gradients([rows, rows, 4], [2, 0, 9], 4, 2, 64, rows)
    assert (dq[:rows - 2] == 0).all() and (dq[rows:2 * rows] == 0).all()


@pytest.mark.gpu
def test_no_queries_and_no_keys():
    for ql, kl in (([0, 0], [40, 3]), ([9], [0]), ([0], [0])):
        *_, (dq, dk, dv) = gradients(ql, kl, 4, 2, 64, 3)
        assert (dq == 0).all() and (dk == 0).all() and (dv == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,n", [(8, 1, 64, 2048), (1, 1, 128, 3001), (32, 8, 128, 1500)])
def test_long_prompts(Hq, Hkv, D, n):
    """With and without a split of the walked axes."""
    gradients([n], [n], Hq, Hkv, D, n)


@pytest.mark.gpu
def test_many_sequences_strided_tokens_large_scores():
    lens = [int(x) for x in np.random.default_rng(1).integers(0, 12, 200)]
    gradients(lens, lens, 4, 2, 64, 6, pad=24)
    gradients([400], [400], 2, 1, 128, 7, gain=60.0)


@pytest.mark.gpu
@pytest.mark.parametrize("seqs", [5, 45])
@pytest.mark.parametrize("Hq,Hkv,D", [(12, 3, 64), (16, 1, 128)])
def test_tiles_that_lie_across_workgroups(seqs, Hq, Hkv, D):
    """Long and short sequences, few enough to fit the table of sequences and more than that."""
    lens = [int(x) for x in np.random.default_rng(seqs).choice([0, 1, 100, 129, 700, 1300], seqs - 1)] + [1111]
    gradients(lens, [n + 7 * (n > 100) for n in lens], Hq, Hkv, D, seqs)


@pytest.mark.gpu
def test_same_bits_workspace_outputs_and_stream():
    q, k, v, d_o, o, lse, cu, ref = gradients([600, 100], [600, 700], 4, 1, 64, 9)
    nb = K.attend_backward_workspace_bytes(cu[0], cu[2], 4, 1, 64)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        outs = [torch.full((t.shape[0] + 3, *t.shape[1:]), 3.0, dtype=BF16, device="cuda") for t in ref]
        torch.cuda.synchronize()
        K.attend_backward(d_o, q, k, v, o, lse, *cu, workspace=ws, stream=stream,
                          **{n: t[:r.shape[0]] for n, t, r in zip(("dq", "dk", "dv"), outs, ref)})
        torch.cuda.synchronize()
        for t, r in zip(outs, ref):
            assert torch.equal(t[:r.shape[0]], r) and (t[r.shape[0]:] == 3.0).all()


@pytest.mark.gpu
def test_gradients_match_differences():
    """Along random directions, against central differences of the 64-bit attention.  The
    kernel's gradients are off by about h = 2^-8 of the terms' magnitudes (o, P, dS and the
    outputs are rounded to bf16, 4 roundings), the differences by about 1e-8."""
    n, Hq, Hkv, D = 70, 4, 2, 64
    q, k, v, d_o, o, lse, cu, (dq, dk, dv) = gradients([n], [n], Hq, Hkv, D, 5)
    seen = torch.ones(n, n, device="cuda").tril() > 0

    def loss(q, k, v):
        kk, vv = k.repeat_interleave(Hq // Hkv, 1), v.repeat_interleave(Hq // Hkv, 1)
        s = torch.stack([q[:, h] @ kk[:, h].t() for h in range(Hq)]) / D ** 0.5
        p = torch.softmax(s.masked_fill(~seen, -float("inf")), 2)
        return (torch.stack([p[h] @ vv[:, h] for h in range(Hq)], 1) * d_o.double()).sum()

    x = [t[:n].double() for t in (q, k, v)]
    g = torch.Generator().manual_seed(2)
    for i, grad in enumerate((dq, dk, dv)):
        d = torch.randn(x[i].shape, generator=g, dtype=torch.float64).cuda()
        up, dn = list(x), list(x)
        up[i], dn[i] = x[i] + 1e-5 * d, x[i] - 1e-5 * d
        num = (loss(*up) - loss(*dn)) / 2e-5
        terms = grad.double() * d
        assert abs(num - terms.sum()) <= 4 * 2.0 ** -8 * terms.abs().sum()


@pytest.mark.gpu
def test_captured_step_replays_equal_eager():
    cu_q, cqd = cu_of([300, 40])
    q, k, v = make(cu_q, cu_q, 4, 1, 64, 12)
    d_o = torch.randn(340, 4, 64, generator=torch.Generator().manual_seed(3)).to(BF16).cuda()

    def step():
        o, lse = K.attend(q, k, v, cu_q, cqd, want_lse=True)
        return (o, lse) + K.attend_backward(d_o, q, k, v, o, lse, cu_q, cqd)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        q.copy_(make(cu_q, cu_q, 4, 1, 64, 50 + i)[0])
        for t in out:
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(x, y) for x, y in zip(got, step()))


# ---------------------------------------------------------------------------
# Refusals (no GPU)
# ---------------------------------------------------------------------------

def _call(**kw):
    a = dict(d_o=16, q=16, qs=512, k=16, ks=128, v=16, vs=128, o=16, lse=16, cu_q=[0, 4, 6],
             cu_k=[0, 100, 200], cqd=16, ckd=16, nseq=2, Hq=4, Hkv=1, D=128, scale=0.1, ws=16, nb=1 << 40,
             dq=16, dk=16, dv=16)
    a.update(kw)
    cu_q, cu_k = (np.array(a[n], dtype=np.int32) for n in ("cu_q", "cu_k"))
    p = lambda x: x.ctypes.data_as(ctypes.c_void_p)
    return K.lib().kpool_attend_backward(
        a["d_o"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["o"], a["lse"], p(cu_q), a["cqd"],
        p(cu_k), a["ckd"], a["nseq"], a["Hq"], a["Hkv"], a["D"], a["scale"], a["ws"], a["nb"], a["dq"],
        a["dk"], a["dv"], None)


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, K.KPOOL_EINVAL) for n in ("d_o", "q", "k", "v", "o", "lse", "cqd", "ckd", "dq", "dk", "dv")],
    *[({n: 24}, K.KPOOL_EINVAL) for n in ("d_o", "q", "k", "v", "o", "dq", "dk", "dv", "ws")],
    (dict(lse=18), K.KPOOL_EINVAL), (dict(ws=None), K.KPOOL_EWORKSPACE), (dict(nb=100), K.KPOOL_EWORKSPACE),
    (dict(cu_q=[0, 5, 4]), K.KPOOL_EINVAL), (dict(Hkv=3), K.KPOOL_EINVAL), (dict(D=20), K.KPOOL_EINVAL),
    (dict(D=256), K.KPOOL_EUNSUPPORTED), (dict(scale=0.0), K.KPOOL_EINVAL), (dict(qs=500), K.KPOOL_EINVAL),
    (dict(cu_q=[0, 0, 0], cqd=None), K.KPOOL_EINVAL), (dict(cu_q=[0, 0, 0], dk=None), K.KPOOL_EINVAL),
])
def test_refuses(kw, code):
    assert _call(**kw) == code
    assert K.lib().kpool_last_error()


def test_nothing_to_do_needs_no_pointers():
    none = {n: None for n in ("d_o", "q", "k", "v", "o", "lse", "cqd", "ckd", "ws", "dq", "dk", "dv")}
    assert _call(cu_q=[0, 0, 0], cu_k=[0, 0, 0], **none) == K.KPOOL_OK


def test_workspace_bytes():
    nb = K.attend_backward_workspace_bytes([0, 4, 6], [0, 100, 200], 4, 1, 128)
    assert nb >= 6 * 4 * 8
    assert _call(nb=nb - 1) == K.KPOOL_EWORKSPACE
    assert K.attend_backward_workspace_bytes([0, 0], [0, 5], 4, 1, 128) == 0
    with pytest.raises(K.KpoolError):
        K.attend_backward_workspace_bytes([0, 4], [0, 4], 4, 3, 128)


APART = dict(d_o=1 << 20, q=2 << 20, k=3 << 20, v=4 << 20, o=5 << 20, lse=6 << 20, ws=7 << 20, dq=8 << 20,
             dk=9 << 20, dv=10 << 20)


@pytest.mark.parametrize("kw", [
    *[{out: APART[n]} for out in ("dq", "dk", "dv") for n in ("d_o", "q", "k", "v", "o", "lse")],
    dict(dk=APART["dv"]), dict(dq=APART["dk"]), dict(dv=APART["dq"] + 16),
    dict(dk=APART["k"] + 199 * 256), dict(dq=APART["d_o"] - 16)])
def test_refuses_outputs_over_inputs(kw):
    assert _call(**{**APART, **kw}) == K.KPOOL_EINVAL
    assert b"overlaps" in K.lib().kpool_last_error()


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=24), dict(v=24)])
def test_keys_without_rows_need_their_pointers(kw):
    """The keys' kernel loads its keys even where no row sees them."""
    assert _call(**{**APART, "cu_q": [0, 0, 0], **kw}) == K.KPOOL_EINVAL


@pytest.mark.parametrize("kw", [
    *[dict(ws=APART[n]) for n in ("d_o", "q", "k", "v", "o", "lse", "dq", "dk", "dv")],
    *[{out: 11 << 20, n: 11 << 20} for out in ("ws", "dq", "dk", "dv") for n in ("cqd", "ckd")]])
def test_refuses_a_workspace_over_operands_and_outputs_over_lengths(kw):
    assert _call(**{**APART, "cqd": 12 << 20, "ckd": 13 << 20, **kw}) == K.KPOOL_EINVAL
    assert b"overlaps" in K.lib().kpool_last_error()


@pytest.mark.parametrize("nseq,code", [(1 << 17, K.KPOOL_EINVAL), (1 << 18, K.KPOOL_EUNSUPPORTED)])
def test_refuses_more_sequences_than_the_sum_of_parts_takes(nseq, code):
    """Few rows among very many empty sequences: eight workgroups a tile add dQ's parts."""
    cu_q, cu_k = np.zeros((2, nseq + 1), dtype=np.int32)
    cu_q[6:], cu_k[6:] = 64, 500
    at = dict(d_o=1 << 40, q=2 << 40, k=3 << 40, v=4 << 40, o=5 << 40, lse=6 << 40, ws=7 << 40, dq=2 << 40,
              dk=9 << 40, dv=10 << 40, cqd=11 << 40, ckd=12 << 40)
    assert _call(**at, cu_q=cu_q, cu_k=cu_k, nseq=nseq, Hq=8, Hkv=8, qs=1024, ks=1024, vs=1024, nb=1 << 60) == code


@pytest.mark.parametrize("name", ["cqd", "ckd"])
def test_refuses_lengths_off_their_elements(name):
    assert _call(**{**APART, "cqd": 12 << 20, "ckd": 13 << 20, name: (13 << 20) + 1}) == K.KPOOL_EINVAL
    assert b"aligned" in K.lib().kpool_last_error()
