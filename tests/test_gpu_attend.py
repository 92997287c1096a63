"""kpool_attend and kpool_attend_selected against attention in 64 bits (tolerances:
attend_reference.py)."""
import ctypes

import numpy as np
import pytest
import torch

from attend_reference import check, cu_of, make
from pool_score_top_amd import kpool as K

BF16 = torch.bfloat16


def run(q_lens, k_lens, Hq, Hkv, D, seed, pad=0, gain=2.0):
    cu_q, cqd = cu_of(q_lens)
    cu_k, ckd = cu_of(k_lens)
    q, k, v = make(cu_q, cu_k, Hq, Hkv, D, seed, pad, gain)
    o, lse = K.attend(q, k, v, cu_q, cqd, cu_k, ckd, want_lse=True)
    check(q, k, v, cu_q, cu_k, 1.0 / D ** 0.5, o, lse)
    return q, k, v, (cu_q, cqd, cu_k, ckd), o, lse


# ---------------------------------------------------------------------------
# Whole keys
# ---------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 8), (4, 4, 16), (4, 1, 64), (8, 2, 72), (6, 2, 128),
                                      (5, 1, 120), (32, 1, 128), (40, 1, 64)])
def test_packed_prompts(Hq, Hkv, D):
    """Lengths around the tiles' edges, an empty sequence, a single token."""
    lens = [1, 31, 0, 32, 33, 63, 64, 65, 257, 300, 2]
    run(lens, lens, Hq, Hkv, D, Hq * 1000 + D)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 128), (12, 4, 64), (16, 1, 128)])
def test_chunks_of_prompts(Hq, Hkv, D):
    """Queries at the end of longer keys: a few rows, many rows, none."""
    run([5, 100, 0, 1, 260], [50, 1000, 77, 4096, 261], Hq, Hkv, D, Hq + D)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 8, 64), (32, 4, 128), (7, 1, 80), (64, 1, 128)])
@pytest.mark.parametrize("keys", [[1], [517], [33, 1, 2048, 5000, 129], [30000, 3]])
def test_single_tokens(Hq, Hkv, D, keys):
    """One new token a sequence, with and without a split of the key axis."""
    run([1] * len(keys), keys, Hq, Hkv, D, Hq + D + len(keys))


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 300])
def test_rows_without_keys(rows):
    """More queries than keys: the first rows see nothing; a sequence without any key."""
    run([rows, rows, 4], [2, 0, 9], 4, 2, 64, rows)


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens,k_lens", [([200], [200]), ([1, 1], [900, 3000])])
def test_strided_tokens(q_lens, k_lens):
    run(q_lens, k_lens, 8, 2, 128, 4, pad=24)


@pytest.mark.gpu
def test_long_prompt_and_many_sequences():
    run([3000], [3000], 4, 1, 128, 5)
    lens = [int(x) for x in np.random.default_rng(1).integers(0, 12, 200)]
    run(lens, lens, 4, 2, 64, 6)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [([700], [700]), ([1], [4000])])
def test_scores_of_every_size(lens):
    """Large scores (one key takes all the weight), tiny ones (all keys alike), and a maximum
    that rises with every key, which moves the running maximum all the way."""
    run(*lens, 2, 1, 128, 7, gain=60.0)
    run(*lens, 2, 1, 128, 8, gain=1e-3)
    cu_q, cqd = cu_of(lens[0])
    cu_k, ckd = cu_of(lens[1])
    n = int(cu_k[-1])
    q = torch.full((int(cu_q[-1]), 2, 64), 1.0, dtype=BF16, device="cuda")
    k = (torch.arange(n, device="cuda") / 16).to(BF16)[:, None, None].expand(n, 1, 64).contiguous()
    for sign in (1.0, -1.0):
        v = torch.randn(n, 1, 64, generator=torch.Generator().manual_seed(9)).to(BF16).cuda()
        o, lse = K.attend(q, k * sign, v, cu_q, cqd, cu_k, ckd, want_lse=True)
        check(q, k * sign, v, cu_q, cu_k, 0.125, o, lse)


@pytest.mark.gpu
def test_same_bits_other_stream_workspace_and_outputs():
    q, k, v, cu, o, lse = run([1, 1], [9000, 20000], 16, 2, 128, 10)
    nb = K.attend_workspace_bytes(cu[0], cu[2], 16, 2, 128)
    assert nb > 0
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        ws.fill_(255)
        torch.cuda.synchronize()
        big = torch.full((5, 16, 128), 3.0, dtype=BF16, device="cuda")
        l2 = torch.empty_like(lse)
        torch.cuda.synchronize()
        o2, _ = K.attend(q, k, v, *cu, out=big[:2], lse=l2, workspace=ws, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(o2, o) and torch.equal(l2, lse) and (big[2:] == 3.0).all()
    q, k, v, cu, o, lse = run([500, 40], [500, 900], 4, 2, 128, 11)
    bits = lambda t: t.view(torch.int16)
    o2, none = K.attend(bits(q), bits(k), bits(v), *cu)
    assert none is None and torch.equal(o2, bits(o))


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["rows", "tiles", "selected"])
def test_captured_calls_replay_equal_eager(form):
    q_lens, k_lens = ([400, 30], [400, 2000]) if form == "tiles" else ([1, 1, 1], [4000, 9000, 7])
    cu_q, cqd = cu_of(q_lens)
    cu_k, ckd = cu_of(k_lens)
    q, k, v = make(cu_q, cu_k, 8, 2, 128, 12)
    ids = torch.randint(-1, 4000, (int(cu_q[-1]), 600), generator=torch.Generator().manual_seed(1),
                        dtype=torch.int32).cuda()
    call = lambda: (K.attend_selected(q, k, v, ids, cu_q, cqd, cu_k, ckd, want_lse=True)
                    if form == "selected" else K.attend(q, k, v, cu_q, cqd, cu_k, ckd, want_lse=True))
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        q.copy_(make(cu_q, cu_k, 8, 2, 128, 50 + i)[0])
        for t in out:
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(x, y) for x, y in zip(got, call()))


# ---------------------------------------------------------------------------
# Selected tokens
# ---------------------------------------------------------------------------

def lists(cu_q, cu_k, width, seed, kind):
    """Ids per row: random ones, absent entries among them, ids before 0 and past the row, the
    same id more than once, rows with none at all."""
    g = torch.Generator().manual_seed(seed)
    rows = int(cu_q[-1])
    t = np.concatenate([np.arange(d - c - (b - a), d - c) for a, b, c, d in
                        zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:])] or [np.zeros(0)])
    t = torch.from_numpy(t.astype(np.int64))
    r = torch.rand(rows, width, generator=g)
    ids = (r * (t[:, None].clamp(min=0) + 1)).long()
    if kind == "full":
        return ids.to(torch.int32).cuda()
    ids[torch.rand(rows, width, generator=g) < 0.4] = -1
    ids[torch.rand(rows, width, generator=g) < 0.05] = -2 ** 31
    ids[torch.rand(rows, width, generator=g) < 0.05] = 2 ** 31 - 1
    past = torch.rand(rows, width, generator=g) < 0.1
    ids = torch.where(past, t[:, None] + 1, ids)
    ids[::7] = -1
    if width > 40:
        ids[1::7, 33:] = -1   # a tile and a half
        ids[2::7, :width - 3] = -1
    return ids.to(torch.int32).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["full", "ragged"])
@pytest.mark.parametrize("Hq,Hkv,D,width", [(1, 1, 8, 1), (4, 4, 16, 16), (8, 2, 64, 100), (16, 1, 128, 257),
                                            (6, 2, 128, 31), (40, 1, 64, 32), (70, 2, 80, 130),
                                            (32, 2, 128, 2048)])
def test_selected_tokens(Hq, Hkv, D, width, kind):
    q_lens, k_lens = [40, 1, 0, 9, 3], [40, 700, 5, 3000, 2]
    cu_q, cqd = cu_of(q_lens)
    cu_k, ckd = cu_of(k_lens)
    q, k, v = make(cu_q, cu_k, Hq, Hkv, D, Hq + width, pad=8 if D == 128 else 0)
    ids = lists(cu_q, cu_k, width, 3, kind)
    o, lse = K.attend_selected(q, k, v, ids, cu_q, cqd, cu_k, ckd, want_lse=True)
    check(q, k, v, cu_q, cu_k, 1.0 / D ** 0.5, o, lse, ids)
    o2, _ = K.attend_selected(q, k, v, ids, cu_q, cqd, cu_k, ckd)
    assert torch.equal(o, o2)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [1, 300, 2048])
def test_selected_single_token_and_no_width(width):
    cu_q, cqd = cu_of([1])
    cu_k, ckd = cu_of([50000])
    q, k, v = make(cu_q, cu_k, 8, 1, 128, width)
    ids = lists(cu_q, cu_k, width, 5, "full")
    o, lse = K.attend_selected(q, k, v, ids, cu_q, cqd, cu_k, ckd, want_lse=True)
    check(q, k, v, cu_q, cu_k, 1.0 / 128 ** 0.5, o, lse, ids)
    o, lse = K.attend_selected(q, k, v, ids[:, :0].contiguous(), cu_q, cqd, cu_k, ckd, want_lse=True)
    assert (o == 0).all() and (lse == -float("inf")).all()


@pytest.mark.gpu
def test_selected_reads_listed_tokens_only():
    """NaN and infinities in every key and value that no list names leave no trace."""
    cu_q, cqd = cu_of([30, 2])
    cu_k, ckd = cu_of([900, 400])
    q, k, v = make(cu_q, cu_k, 8, 2, 128, 21)
    ids = lists(cu_q, cu_k, 64, 6, "ragged")
    o, lse = K.attend_selected(q, k, v, ids, cu_q, cqd, cu_k, ckd, want_lse=True)
    used = torch.zeros(1302, dtype=torch.bool, device="cuda")
    for a, b, c, d in ((0, 30, 0, 900), (30, 32, 900, 1300)):
        t = torch.arange(d - c - (b - a), d - c, device="cuda")[:, None]
        x = ids[a:b].long()
        used[c + x[(x >= 0) & (x <= t)]] = True
    k, v = k.clone(), v.clone()
    k[~used], v[~used] = float("nan"), float("inf")
    o2, lse2 = K.attend_selected(q, k, v, ids, cu_q, cqd, cu_k, ckd, want_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


# ---------------------------------------------------------------------------
# Refusals (no GPU: the checks come before any launch)
# ---------------------------------------------------------------------------

def _call(selected, **kw):
    a = dict(q=16, qs=512, k=16, ks=128, v=16, vs=128, ids=16, width=8, cu_q=[0, 4, 6], cu_k=[0, 100, 200],
             cqd=16, ckd=16, nseq=2, Hq=4, Hkv=1, D=128, scale=0.1, ws=16, nb=1 << 40, o=16, lse=16)
    a.update(kw)
    cu_q, cu_k = (np.array(a[n], dtype=np.int32) if a[n] is not None else None for n in ("cu_q", "cu_k"))
    p = lambda x: None if x is None else x.ctypes.data_as(ctypes.c_void_p)
    rows = (a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"])
    rest = (p(cu_q), a["cqd"], p(cu_k), a["ckd"], a["nseq"], a["Hq"], a["Hkv"], a["D"], a["scale"], a["ws"],
            a["nb"], a["o"], a["lse"], None)
    if selected:
        return K.lib().kpool_attend_selected(*rows, a["ids"], a["width"], *rest)
    return K.lib().kpool_attend(*rows, *rest)


BAD = [
    (dict(q=None), K.KPOOL_EINVAL), (dict(k=None), K.KPOOL_EINVAL), (dict(v=None), K.KPOOL_EINVAL),
    (dict(o=None), K.KPOOL_EINVAL), (dict(cqd=None), K.KPOOL_EINVAL), (dict(ckd=None), K.KPOOL_EINVAL),
    (dict(q=24), K.KPOOL_EINVAL), (dict(k=24), K.KPOOL_EINVAL), (dict(v=24), K.KPOOL_EINVAL),
    (dict(o=24), K.KPOOL_EINVAL), (dict(lse=18), K.KPOOL_EINVAL),
    (dict(qs=504), K.KPOOL_EINVAL), (dict(qs=516), K.KPOOL_EINVAL), (dict(ks=120), K.KPOOL_EINVAL),
    (dict(vs=1 << 25), K.KPOOL_EINVAL), (dict(cu_q=None), K.KPOOL_EINVAL), (dict(cu_k=None), K.KPOOL_EINVAL),
    (dict(cu_q=[1, 4, 6]), K.KPOOL_EINVAL), (dict(cu_k=[0, 100, 99]), K.KPOOL_EINVAL),
    (dict(nseq=0), K.KPOOL_EINVAL), (dict(Hq=0), K.KPOOL_EINVAL), (dict(Hkv=0), K.KPOOL_EINVAL),
    (dict(Hkv=3), K.KPOOL_EINVAL), (dict(D=0), K.KPOOL_EINVAL), (dict(D=12), K.KPOOL_EINVAL),
    (dict(D=136), K.KPOOL_EUNSUPPORTED), (dict(scale=0.0), K.KPOOL_EINVAL),
    (dict(scale=float("nan")), K.KPOOL_EINVAL), (dict(scale=float("inf")), K.KPOOL_EINVAL),
    (dict(cu_q=[0, 1 << 30, 1 << 30], cu_k=[0, 1 << 30, 1 << 30]), K.KPOOL_EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD)
@pytest.mark.parametrize("selected", [False, True])
def test_refuses(selected, kw, code):
    assert _call(selected, **kw) == code
    assert K.lib().kpool_last_error()


@pytest.mark.parametrize("kw,code", [(dict(width=-1), K.KPOOL_EINVAL), (dict(ids=None), K.KPOOL_EINVAL),
                                     (dict(ids=18), K.KPOOL_EINVAL)])
def test_selected_refuses(kw, code):
    assert _call(True, **kw) == code


def test_workspace_sizes_and_refusals():
    one = dict(cu_q=[0, 1, 2], cu_k=[0, 50000, 100000])
    nb = K.attend_workspace_bytes([0, 1, 2], [0, 50000, 100000], 4, 1, 128)
    assert nb > 0 and nb % (2 * 4 * 129 * 4) == 0
    assert _call(False, **one, nb=nb - 1) == K.KPOOL_EWORKSPACE
    assert _call(False, **one, ws=None) == K.KPOOL_EWORKSPACE
    assert _call(False, **one, ws=24) == K.KPOOL_EINVAL
    assert K.attend_workspace_bytes([0, 9000], [0, 9000], 32, 8, 128) == 0
    nb = K.attend_selected_workspace_bytes(2, 2, 2048, 4, 1, 128)
    assert nb > 0
    assert _call(True, **one, width=2048, nb=nb - 1) == K.KPOOL_EWORKSPACE
    assert K.attend_selected_workspace_bytes(4096, 1, 2048, 4, 1, 128) == 0
    with pytest.raises(K.KpoolError):
        K.attend_workspace_bytes([0, 5, 3], [0, 5, 5], 4, 1, 128)
    with pytest.raises(K.KpoolError):
        K.attend_selected_workspace_bytes(2, 2, 2048, 4, 3, 128)


def test_no_queries_need_no_pointers():
    none = dict(cu_q=[0, 0, 0], q=None, k=None, v=None, o=None, cqd=None, ckd=None, ws=None, lse=None)
    assert _call(False, **none) == K.KPOOL_OK
    assert _call(True, **none, ids=None) == K.KPOOL_OK


@pytest.mark.gpu
def test_binding_refuses():
    cu, cud = cu_of([4])
    t = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device="cuda")
    q, k = t(4, 4, 64), t(4, 2, 64)
    ids = t(4, 8, dtype=torch.int32)
    bad = [
        lambda: K.attend(q.half(), k, k, cu, cud), lambda: K.attend(q.cpu(), k, k, cu, cud),
        lambda: K.attend(q, k.cpu(), k, cu, cud), lambda: K.attend(q, t(4, 2, 32), k, cu, cud),
        lambda: K.attend(q, k, t(4, 1, 64), cu, cud), lambda: K.attend(q[:3], k, k, cu, cud),
        lambda: K.attend(q, k[:3], k, cu, cud), lambda: K.attend(q, k, k, cu, cud.cpu()),
        lambda: K.attend(q, k, k, cu, cud, cu), lambda: K.attend(q, k, k, cu, cud[:1]),
        lambda: K.attend(q.transpose(1, 2), k, k, cu, cud), lambda: K.attend(q, k, k, cu, cud.long()),
        lambda: K.attend(q, k, k, cu, cud, out=t(5, 4, 64)), lambda: K.attend(q, k, k, cu, cud, lse=t(4, 4)),
        lambda: K.attend_selected(q, k, k, ids[:3], cu, cud),
        lambda: K.attend_selected(q, k, k, ids.long(), cu, cud),
        lambda: K.attend_selected(q, k, k, ids[:, ::2], cu, cud),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(K.KpoolError):
        K.attend(q, k, k, cu, cud, scale=-1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 8, 64), (40, 4, 128), (3, 1, 16)])
def test_selected_many_rows(Hq, Hkv, D):
    """Enough rows for a wave each; lists of several blocks of 1024 entries."""
    q_lens, k_lens = [1500, 0, 700], [1500, 3, 4000]
    cu_q, cqd = cu_of(q_lens)
    cu_k, ckd = cu_of(k_lens)
    q, k, v = make(cu_q, cu_k, Hq, Hkv, D, 31)
    for width, kind in ((130, "ragged"), (2100, "full")):
        ids = lists(cu_q, cu_k, width, 3, kind)
        o, lse = K.attend_selected(q, k, v, ids, cu_q, cqd, cu_k, ckd, want_lse=True)
        check(q, k, v, cu_q, cu_k, 1.0 / D ** 0.5, o, lse, ids)
        assert torch.equal(o, K.attend_selected(q, k, v, ids, cu_q, cqd, cu_k, ckd)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(17, 1, 128), (64, 2, 64), (32, 2, 120)])
def test_selected_many_rows_of_many_heads(Hq, Hkv, D):
    """A wave a row with more than 16 heads a key head, and with exactly 16."""
    cu_q, cqd = cu_of([100, 950])
    cu_k, ckd = cu_of([131, 3000])
    q, k, v = make(cu_q, cu_k, Hq, Hkv, D, 33)
    for width, kind in ((97, "ragged"), (2049, "full")):
        ids = lists(cu_q, cu_k, width, 5, kind)
        o, lse = K.attend_selected(q, k, v, ids, cu_q, cqd, cu_k, ckd, want_lse=True)
        check(q, k, v, cu_q, cu_k, 1.0 / D ** 0.5, o, lse, ids)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("keys", [65536, 65537, 70001])
def test_selected_around_the_16_bit_ids(keys, D):
    """Sequences whose ids just fit 16 bits and just do not; the last ids are in every list."""
    cu_q, cqd = cu_of([1030])
    cu_k, ckd = cu_of([keys])
    q, k, v = make(cu_q, cu_k, 2, 1, D, 35)
    ids = lists(cu_q, cu_k, 1500, 7, "full")
    t = torch.arange(keys - 1030, keys, device="cuda", dtype=torch.int32)
    ids[:, 3], ids[:, 1400], ids[:, 1025] = t, t - 1, 0
    o, lse = K.attend_selected(q, k, v, ids, cu_q, cqd, cu_k, ckd, want_lse=True)
    check(q, k, v, cu_q, cu_k, 1.0 / D ** 0.5, o, lse, ids)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 1100])
def test_selected_one_token_over_and_over(rows):
    """All of a list in one place; and all its tokens but one there."""
    cu_q, cqd = cu_of([rows])
    cu_k, ckd = cu_of([5000])
    q, k, v = make(cu_q, cu_k, 4, 1, 128, 37)
    for last in (7, 3000):
        ids = torch.full((rows, 4100), 7, dtype=torch.int32, device="cuda")
        ids[:, 4099] = last
        o, lse = K.attend_selected(q, k, v, ids, cu_q, cqd, cu_k, ckd, want_lse=True)
        check(q, k, v, cu_q, cu_k, 1.0 / 128 ** 0.5, o, lse, ids)


@pytest.mark.gpu
def test_more_sequences_than_the_table():
    """Tokens, chunks and lists of 70 sequences, some empty (found by search on the device)."""
    rng = np.random.default_rng(4)
    k_lens = [int(x) for x in rng.integers(0, 300, 70)]
    for q_lens in ([min(1, n) for n in k_lens], [int(rng.integers(0, n + 1)) for n in k_lens]):
        q, k, v, cu, o, lse = run(q_lens, k_lens, 4, 2, 64, 8)
        ids = lists(cu[0], cu[2], 40, 5, "ragged")
        o, lse = K.attend_selected(q, k, v, ids, *cu, want_lse=True)
        check(q, k, v, cu[0], cu[2], 0.125, o, lse, ids)


@pytest.mark.gpu
@pytest.mark.parametrize("keys", [[300], [9000]])
def test_nan_in_a_query_stays_in_its_row(keys):
    """Inputs have to be finite; a row that is not still gives NaN, with and without a split,
    and spoils no other row."""
    cu_q, cqd = cu_of([2])
    cu_k, ckd = cu_of(keys)
    q, k, v = make(cu_q, cu_k, 4, 1, 64, 3)
    ref, ref_lse = K.attend(q, k, v, cu_q, cqd, cu_k, ckd, want_lse=True)
    q = q.clone()
    q[1, 2, 5] = float("nan")
    o, lse = K.attend(q, k, v, cu_q, cqd, cu_k, ckd, want_lse=True)
    assert o[1, 2].isnan().all() and lse[1, 2].isnan()
    keep = torch.ones(2, 4, dtype=torch.bool, device="cuda")
    keep[1, 2] = False
    assert torch.equal(o[keep], ref[keep]) and torch.equal(lse[keep], ref_lse[keep])


APART = dict(q=1 << 20, k=2 << 20, v=3 << 20, ids=4 << 20, ws=5 << 20, o=6 << 20, lse=7 << 20)


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("kw", [
    *[{out: APART[n]} for out in ("o", "lse") for n in ("q", "k", "v")], dict(lse=APART["o"]),
    dict(o=APART["k"] + 199 * 256), dict(o=APART["q"] - 16), dict(o=APART["q"] + 6 * 1024 - 16)])
def test_refuses_outputs_over_inputs(selected, kw):
    assert _call(selected, **{**APART, **kw}) == K.KPOOL_EINVAL
    assert b"overlaps" in K.lib().kpool_last_error()


@pytest.mark.parametrize("out", ["o", "lse"])
def test_refuses_outputs_over_lists(out):
    assert _call(True, **{**APART, out: APART["ids"]}) == K.KPOOL_EINVAL
    assert b"overlaps" in K.lib().kpool_last_error()


@pytest.mark.gpu
def test_outputs_in_the_gaps_of_strided_inputs():
    """What lies between the rows of a strided input is not the input's."""
    cu, dev = cu_of([1])
    ck, ckd = cu_of([40])
    q, k, v = make(cu, ck, 2, 1, 64, 4)
    ref, _ = K.attend(q, k, v, cu, dev, ck, ckd)
    buf = torch.zeros(40, 256, dtype=torch.bfloat16, device="cuda")
    buf[:, :64], buf[:, 64:128] = k[:40, 0], v[:40, 0]
    out = buf[7, 128:].view(1, 2, 64)
    K.attend(q, buf[:, None, :64], buf[:, None, 64:128], cu, dev, ck, ckd, out=out)
    assert torch.equal(out, ref)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Tokens 2^24 elements apart (the widest stride), 10 GB of them: the same bits as from tokens
    side by side, by every kernel; the layer norm's rows likewise."""
    T, wide = 300, 1 << 24
    cu, dev = cu_of([T])
    one, one_dev = cu_of([1])
    q, k, v = (t[:T] for t in make(cu, cu, 4, 2, 64, 41))
    far = torch.empty(T * wide, dtype=BF16, device="cuda").view(T, wide)
    fq, fk, fv = (far[:, at:at + t[0].numel()].unflatten(1, t.shape[1:]) for at, t in ((0, q), (256, k), (wide - 128, v)))
    for f, t in ((fq, q), (fk, k), (fv, v)):
        f.copy_(t)
    q, k, v = (t.contiguous() for t in (q, k, v))
    ids = lists(cu, cu, 70, 3, "ragged")
    many = torch.arange(T, dtype=torch.int32, device="cuda").repeat(T, 4)
    d_o = torch.randn(T, 4, 64, device="cuda").to(BF16)

    def calls(q, k, v):
        o, lse = K.attend(q, k, v, cu, dev, want_lse=True)
        out = [o, lse, *K.attend_backward(d_o, q, k, v, o, lse, cu, dev)]
        out += K.attend(q[T - 1:], k, v, one, one_dev, cu, dev, want_lse=True)
        for lists_of in (ids, many):
            out += K.attend_selected(q, k, v, lists_of, cu, dev, want_lse=True)
        return out + [K.layer_norm(x.flatten(1))[0] for x in (k, v)]

    for near, there in zip(calls(q, k, v), calls(fq, fk, fv)):
        assert torch.equal(near, there)


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("name", ["q", "k", "v", "o", "lse", "cqd", "ckd", "ids"])
def test_refuses_a_workspace_over_operands(selected, name):
    """Single tokens over long keys, whose parts take a workspace."""
    if name == "ids" and not selected:
        return
    at = dict(q=1 << 32, k=2 << 32, v=3 << 32, ids=4 << 32, ws=5 << 32, o=6 << 32, lse=7 << 32, cqd=8 << 32,
              ckd=9 << 32)
    at["ws"] = at[name] if name in ("cqd", "ckd") else at[name] + 16
    assert _call(selected, **at, cu_q=[0, 1, 2], cu_k=[0, 50000, 100000], width=2048) == K.KPOOL_EINVAL
    assert b"overlaps" in K.lib().kpool_last_error()


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("out", ["o", "lse"])
@pytest.mark.parametrize("name", ["cqd", "ckd"])
def test_refuses_outputs_over_lengths(selected, out, name):
    at = dict(APART, cqd=8 << 20, ckd=9 << 20)
    at[out] = at[name]
    assert _call(selected, **at) == K.KPOOL_EINVAL
    assert b"overlaps" in K.lib().kpool_last_error()


def _codes(selected, lens_q, lens_k, **kw):
    """What a call answers whose outputs overlap its inputs: that refusal comes last."""
    cu = lambda lens: np.concatenate([[0], np.cumsum(lens)])
    at = dict(q=1 << 40, k=2 << 40, v=3 << 40, ids=4 << 40, ws=5 << 40, o=1 << 40, lse=None, cqd=8 << 40, ckd=9 << 40)
    return _call(selected, **{**at, "nb": 1 << 60, "cu_q": cu(lens_q), "cu_k": cu(lens_k), "nseq": len(lens_q), **kw})


def test_takes_as_many_rows_as_a_launch_holds():
    """Lists of many rows go four to a workgroup: 524288 rows of 32 key heads are 2^22 workgroups."""
    kw = dict(Hkv=32, ks=4096, vs=4096, width=64)
    assert _codes(True, [524288], [524288], Hq=32, qs=4096, **kw) == K.KPOOL_EINVAL
    assert b"overlaps" in K.lib().kpool_last_error()
    assert _codes(True, [1 << 21], [1 << 21], Hq=32, qs=4096, **kw) == K.KPOOL_EUNSUPPORTED
    assert _codes(True, [(1 << 21) - 33], [1 << 21], Hq=32, qs=4096, **kw) == K.KPOOL_EINVAL
    # (and 65 heads a key head are three units)
    assert _codes(True, [1 << 20], [1 << 20], Hq=32 * 65, qs=32 * 65 * 128, **kw) == K.KPOOL_EUNSUPPORTED


@pytest.mark.parametrize("nseq,code", [(1 << 17, K.KPOOL_EINVAL), (1 << 18, K.KPOOL_EUNSUPPORTED)])
def test_refuses_more_sequences_than_the_join_of_parts_takes(nseq, code):
    """Few rows among very many empty sequences: eight workgroups a tile join the parts."""
    lens_q, lens_k = np.zeros((2, nseq), dtype=np.int64)
    lens_q[5], lens_k[5] = 64, 1000
    assert _codes(False, lens_q, lens_k, Hq=8, Hkv=8, qs=1024, ks=1024, vs=1024) == code


@pytest.mark.gpu
def test_selected_rows_of_half_a_million_tokens_and_32_key_heads():
    """2^24 units of work, four to a workgroup."""
    T, H, D = 524288, 32, 8
    cu, dev = cu_of([T])
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(T, H, D, generator=g, device="cuda").to(BF16) for _ in range(3))
    t = torch.arange(T, device="cuda")
    ids = (torch.rand(T, 3, generator=g, device="cuda") * (t[:, None] + 1)).to(torch.int32)
    o, lse = K.attend_selected(q, k, v, ids, cu, dev, want_lse=True)
    rows = torch.cat([t[:50], t[T - 50:], t[::1021]])
    # one sequence a row, its keys the three that it lists
    at = ids[rows].long().flatten()
    n = len(rows)
    cu_q, cu_k = np.arange(n + 1), 3 * np.arange(n + 1)
    three = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda").expand(n, 3)
    check(q[rows], k[at], v[at], cu_q[:201], cu_k[:201], D ** -0.5, o[rows], lse[rows], three)


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("name", ["cqd", "ckd"])
def test_refuses_lengths_off_their_elements(selected, name):
    """Scalar loads would read the word below."""
    assert _call(selected, **{**APART, "cqd": 8 << 20, "ckd": 9 << 20, name: (9 << 20) + 2}) == K.KPOOL_EINVAL
    assert b"aligned" in K.lib().kpool_last_error()
