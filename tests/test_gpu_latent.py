"""kpool_attend_latent and kpool_attend_latent_selected against 64 bits (tolerances:
latent_reference.py)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from attend_reference import cu_of
from latent_reference import BF16, check, lens_of, lists, make
from pool_score_top_amd import kpool as K


def run(q_lens, k_lens, H, R, P, page, seed, width=None, kind="holes", scale=None, **kw):
    q, cache, where, rows = make(q_lens, k_lens, H, R, P, page, seed, **kw)
    cu, dev = cu_of(q_lens)
    scale = (R + P) ** -0.5 if scale is None else scale
    lens = lens_of(k_lens)
    if width is None:
        ids = None
        o, lse = K.attend_latent(q, cache, R, cu, dev, lens, max(k_lens), scale, want_lse=True, **where)
    else:
        ids = lists(q_lens, k_lens, width, seed + 1, kind)
        o, lse = K.attend_latent_selected(q, cache, R, ids, cu, dev, lens, scale, want_lse=True, **where)
    check(q, rows, q_lens, k_lens, R, scale, o, lse, ids)
    return q, cache, where, rows, (cu, dev, lens), ids, o, lse


# heads around the blocks of rows; both compiled widths, odd ones
@pytest.mark.gpu
@pytest.mark.parametrize("H,R,P", [(16, 512, 64), (1, 512, 64), (20, 512, 64), (128, 512, 64), (64, 256, 32),
                                   (5, 8, 8), (33, 264, 0), (16, 128, 64), (100, 504, 40), (16, 40, 0)])
@pytest.mark.parametrize("page", [0, 16])
def test_single_tokens(H, R, P, page):
    """One new token a sequence: lengths around the tiles' and blocks' edges, 1 among them."""
    run([1] * 9, [1, 63, 64, 65, 511, 513, 1025, 130, 2], H, R, P, page, H + R + P)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [1, 7, 64, 100, 1000])
def test_pages(page):
    run([1, 1, 1], [1000, 3, 640], 16, 512, 64, page, page)


@pytest.mark.gpu
@pytest.mark.parametrize("H,page", [(16, 0), (20, 64), (128, 16), (3, 5)])
def test_several_tokens(H, page):
    """A chunk's rows, each up to its own position; no rows, more rows than tokens, no tokens."""
    run([2, 0, 5, 40, 3, 4], [100, 70, 5, 700, 2, 0], H, 512, 64, page, H)


@pytest.mark.gpu
def test_prompts():
    run([300, 77], [300, 1100], 8, 256, 32, 64, 5)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [16, 64])
def test_long_caches(H):
    """Units across many shares, and shares across many units."""
    run([1, 1, 1, 2], [20000, 37, 9001, 300], H, 512, 64, 64, 6)
    run([1], [40000], H, 512, 64, 0, 7)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [16, 40, 64])
@pytest.mark.parametrize("few", [1, 7])
def test_short_units_beside_long_ones(H, few):
    """Shares of several tiles each, and units of fewer tiles than a part of one may have."""
    short = [1, 64, 65, 130, 200, 257, 300, 0, 500]
    run([1] * (2 * len(short) + 2), [40000] + short + [60001] + short, H, 64, 16, 64, 20 + few)
    run([few] * 6, [30000, 130, few, 400, 90000, 65], H, 64, 16, 64, 30)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("width", [1, 128, 200, 256, 300, 500])
def test_short_lists_of_many_rows(H, width):
    run([1100, 0, 33], [1200, 5, 700], H, 64, 16, 64, width, width)


@pytest.mark.gpu
def test_many_sequences():
    """More than a workgroup's threads."""
    g = np.random.default_rng(1)
    q_lens = [int(x) for x in g.integers(0, 3, 700)]
    k_lens = [a + int(x) for a, x in zip(q_lens, g.integers(0, 90, 700))]
    run(q_lens, k_lens, 4, 64, 16, 16, 8)


@pytest.mark.gpu
@pytest.mark.parametrize("H,R,P", [(16, 512, 64), (64, 512, 64), (128, 512, 64), (20, 512, 64), (7, 256, 32), (3, 24, 8)])
@pytest.mark.parametrize("width,kind", [(1, "holes"), (64, "holes"), (700, "holes"), (130, "wild"), (65, "none"),
                                        (600, "all")])
def test_selected(H, R, P, width, kind):
    run([1, 3, 0, 2, 1], [1000, 513, 5, 2, 1], H, R, P, 16 if H % 2 else 0, H + width, width, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [2048, 200])
def test_selected_many_rows(width):
    run([300, 70], [4000, 900], 16, 512, 64, 64, 9, width)


@pytest.mark.gpu
def test_selected_rows_without_tokens():
    run([4, 2], [2, 0], 16, 512, 64, 16, 10, 30, "wild")
    q, cache, where, _, (cu, dev, lens), _, _, _ = run([2], [40], 4, 64, 8, 0, 11)
    ids = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    o, lse = K.attend_latent_selected(q, cache, 64, ids, cu, dev, lens, 0.1, want_lse=True, **where)
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens,H,R,P", [([5, 0, 1, 1, 1], 16, 64, 8), ([5] + [1] * 8, 8, 64, 8), ([33] + [1] * 600, 1, 64, 8),
                                          ([1024], 16, 512, 64), ([2] * 300, 40, 256, 0)])
def test_lists_without_entries(q_lens, H, R, P):
    """Widths of 0 over many rows and sequences: o = 0 and lse = -inf in the workspace that the query names."""
    q, cache, where, _ = make(q_lens, [7] * len(q_lens), H, R, P, 16, 25)
    cu, dev = cu_of(q_lens)
    T = sum(q_lens)
    ids = torch.zeros(T, 0, dtype=torch.int32, device="cuda")
    nb = K.attend_latent_selected_workspace_bytes(T, 0, H, R, P)
    ws = torch.full((max(nb, 1) + 64,), 255, dtype=torch.uint8, device="cuda")
    for workspace in (None, ws[:nb] if nb else None):
        big, lse = torch.full((T + 2, H, R), 3.0, dtype=BF16, device="cuda"), torch.full((T, H), 3.0, device="cuda")
        K.attend_latent_selected(q, cache, R, ids, cu, dev, lens_of([7] * len(q_lens)), 0.1, out=big[:T], lse=lse,
                                 workspace=workspace, **where)
        assert (big[:T] == 0).all() and (big[T:] == 3.0).all() and (lse == -math.inf).all() and (ws[nb:] == 255).all()


@pytest.mark.gpu
@pytest.mark.parametrize("width", [None, 500])
def test_whole_lists_equal_whole_keys_in_64_bits(width):
    """Every token listed in order, beside the whole form: both within the bounds of the same values."""
    run([3], [600], 16, 512, 64, 64, 12, width and 600, "all")


@pytest.mark.gpu
@pytest.mark.parametrize("width", [None, 300])
def test_scores_of_every_size(width):
    for gain in (60.0, 1e-3):
        run([1, 2], [700, 300], 8, 512, 64, 16, 13, width, gain=gain)
    # a maximum that rises with every token, or falls
    n, R, P = 700, 64, 0
    cu, dev = cu_of([1])
    q = torch.ones(1, 4, R, dtype=BF16, device="cuda")
    ids = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    for sign in (1.0, -1.0):
        c = (sign * torch.arange(n, device="cuda") / 16).to(BF16)[:, None].expand(n, R).contiguous()
        where = dict(k_starts=torch.zeros(1, dtype=torch.int32, device="cuda"), want_lse=True)
        if width is None:
            o, lse = K.attend_latent(q, c, R, cu, dev, lens_of([n]), n, 0.125, **where)
        else:
            o, lse = K.attend_latent_selected(q, c, R, ids, cu, dev, lens_of([n]), 0.125, **where)
        check(q, [c], [1], [n], R, 0.125, o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [None, 300])
@pytest.mark.parametrize("page", [0, 16])
def test_strided_tokens_and_rows(width, page):
    run([2, 1], [300, 900], 16, 512, 64, page, 14, width, pad=24)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [None, 400])
def test_tokens_that_the_cache_does_not_have(width):
    """Pages out of range, and rows behind the cache's end or before its start, stand for nothing."""
    q_lens, k_lens, R, P = [2, 1, 1], [400, 300, 50], 256, 32
    cu, dev = cu_of(q_lens)
    for page in (16, 0):
        q, cache, where, rows = make(q_lens, k_lens, 8, R, P, page, 15)
        there = [torch.ones(n, dtype=torch.bool, device="cuda") for n in k_lens]
        if page:
            for s, pg, bad in ((0, 3, -1), (0, 24, cache.shape[0]), (1, 0, 2 ** 31 - 1), (1, 1, -2 ** 31), (2, 0, -1),
                               (2, 1, -3), (2, 2, 1 << 30), (2, 3, -1)):
                where["page_table"][s, pg] = bad
                there[s][pg * page:(pg + 1) * page] = False
        else:
            total = cache.shape[0]
            where["k_starts"][0] = total - 100    # the last 300 tokens lie behind the cache
            where["k_starts"][1] = -1
            where["k_starts"][2] = 2 ** 31 - 10
            rows[0] = torch.cat([cache[total - 100:], rows[0][100:]])
            cache[total - 100:] = torch.randn(100, R + P, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
            rows[0][:100] = cache[total - 100:]
            there[0][100:], there[1][:], there[2][:] = False, False, False
        args = (cu, dev, lens_of(k_lens))
        if width is None:
            ids = None
            o, lse = K.attend_latent(q, cache, R, *args, 400, 0.1, want_lse=True, **where)
        else:
            ids = lists(q_lens, k_lens, width, 3, "wild")
            o, lse = K.attend_latent_selected(q, cache, R, ids, *args, 0.1, want_lse=True, **where)
        check(q, rows, q_lens, k_lens, R, 0.1, o, lse, ids, there)


@pytest.mark.gpu
def test_lengths_are_cut_and_negative_ones_are_none():
    """Lengths past max_len count as max_len, past the table's pages as those, below 0 as 0."""
    R, P, H = 64, 8, 4
    q, cache, where, rows = make([1, 1, 1], [200, 90, 10], H, R, P, 16, 16)
    cu, dev = cu_of([1, 1, 1])
    lens = torch.tensor([2 ** 31 - 1, 90, -5], dtype=torch.int32, device="cuda")
    o, lse = K.attend_latent(q, cache, R, cu, dev, lens, 150, 0.1, want_lse=True, **where)
    check(q, [rows[0][:150], rows[1], rows[2][:0]], [1, 1, 1], [150, 90, 0], R, 0.1, o, lse)
    where["page_table"] = where["page_table"][:, :5].contiguous()   # 80 tokens
    o, lse = K.attend_latent(q, cache, R, cu, dev, lens, 10000, 0.1, want_lse=True, **where)
    check(q, [rows[0][:80], rows[1][:80], rows[2][:0]], [1, 1, 1], [80, 80, 0], R, 0.1, o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [None, 30])
def test_tables_and_caches_of_nothing(width):
    """A page table without columns, a cache without pages or rows: no tokens, o = 0 and lse = -inf."""
    q, cache, where, rows = make([2, 1], [40, 20], 16, 64, 8, 16, 26)
    cu, dev = cu_of([2, 1])
    ids = None if width is None else lists([2, 1], [40, 20], width, 27, "wild")
    none = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    for c, kw in ((cache, dict(page_table=none)), (cache[:0], dict(page_table=none)), (cache[:0], where),
                  (cache.flatten(0, 1)[:0], dict(k_starts=start))):
        if width is None:
            o, lse = K.attend_latent(q, c, 64, cu, dev, lens_of([40, 20]), 40, 0.1, want_lse=True, **kw)
        else:
            o, lse = K.attend_latent_selected(q, c, 64, ids, cu, dev, lens_of([40, 20]), 0.1, want_lse=True, **kw)
        assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.gpu
@pytest.mark.parametrize("width", [None, 600])
def test_same_bits_other_stream_workspace_and_outputs(width):
    q_lens, k_lens, R = [1, 2], [9000, 500], 512
    q, cache, where, _, args, ids, o, lse = run(q_lens, k_lens, 16, R, 64, 64, 17, width)
    scale = 576 ** -0.5
    if width is None:
        nb = K.attend_latent_workspace_bytes(args[0], 9000, 16, R, 64)
        call = lambda **kw: K.attend_latent(q, cache, R, *args, 9000, scale, **where, **kw)
    else:
        nb = K.attend_latent_selected_workspace_bytes(3, width, 16, R, 64)
        call = lambda **kw: K.attend_latent_selected(q, cache, R, ids, *args, scale, **where, **kw)
    assert nb > 0
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        ws.fill_(255)
        big, l2 = torch.full((5, 16, R), 3.0, dtype=BF16, device="cuda"), torch.empty_like(lse)
        torch.cuda.synchronize()
        o2, _ = call(out=big[:3], lse=l2, workspace=ws, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(o2, o) and torch.equal(l2, lse) and (big[3:] == 3.0).all()
    q, cache = q.view(torch.int16), cache.view(torch.int16)
    o2, none = call()
    assert none is None and torch.equal(o2, o.view(torch.int16))


@pytest.mark.gpu
def test_captured_step_replays_while_lengths_and_pages_change():
    """A decoding loop of one captured call: the lengths grow on the device, requests come and go."""
    n, H, R, P, page = 4, 16, 512, 64, 64
    g = torch.Generator().manual_seed(18)
    pages = 200
    cache = torch.randn(pages, page, R + P, generator=g).to(BF16).cuda()
    q = torch.randn(n, H, R + P, generator=g).to(BF16).cuda()
    cu, dev = cu_of([1] * n)
    table = torch.randperm(pages, generator=g)[:n * 50].view(n, 50).to(torch.int32).cuda()
    lens = lens_of([1, 700, 64, 3000])
    call = lambda: K.attend_latent(q, cache, R, cu, dev, lens, 3200, 0.06, page_table=table, want_lse=True)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(5):
        lens.copy_(lens_of([1 + 40 * i, 700 + i, 64 * (i + 1), 0 if i == 2 else 3000 + i]))
        table[1] = table[1].roll(1)
        q.copy_(torch.randn(n, H, R + P, generator=g).to(BF16))
        for t in out:
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, call()))
        k_lens = lens.tolist()
        rows = [cache[table[s, :-(-m // page)].long()].flatten(0, 1)[:m] for s, m in enumerate(k_lens)]
        check(q, rows, [1] * n, k_lens, R, 0.06, *got)


@pytest.mark.gpu
def test_captured_selected_step():
    q, cache, where, rows, args, ids, o, lse = run([1, 2, 1], [700, 300, 1], 64, 512, 64, 16, 19, 400)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = K.attend_latent_selected(q, cache, 512, ids, *args, 576 ** -0.5, want_lse=True, **where)
    for i in range(4):
        new = lists([1, 2, 1], [700, 300, 1], 400, 60 + i, "wild")
        ids.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        ref = K.attend_latent_selected(q, cache, 512, new, *args, 576 ** -0.5, want_lse=True, **where)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.gpu
@pytest.mark.parametrize("width", [None, 300])
def test_nan_in_a_query_stays_in_its_row(width):
    q, cache, where, _, args, ids, ref, ref_lse = run([2], [300], 20, 512, 64, 16, 20, width)
    q = q.clone()
    q[1, 17, 5] = float("nan")
    if width is None:
        o, lse = K.attend_latent(q, cache, 512, *args, 300, 576 ** -0.5, want_lse=True, **where)
    else:
        o, lse = K.attend_latent_selected(q, cache, 512, ids, *args, 576 ** -0.5, want_lse=True, **where)
    assert o[1, 17].isnan().all() and lse[1, 17].isnan()
    keep = torch.ones(2, 20, dtype=torch.bool, device="cuda")
    keep[1, 17] = False
    assert torch.equal(o[keep], ref[keep]) and torch.equal(lse[keep], ref_lse[keep])


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Cache rows 2^24 elements apart, 10 GB of them, and pages far along."""
    n, wide, R, P = 300, 1 << 24, 64, 8
    q, near, where, _ = make([2], [n], 4, R, P, 0, 21)
    start = int(where["k_starts"][0])
    far = torch.empty(n * wide, dtype=BF16, device="cuda").view(n, wide)[:, :R + P]
    far.copy_(near[start:start + n])
    cu, dev = cu_of([2])
    ids = lists([2], [n], 200, 4, "wild")
    zero = dict(k_starts=torch.zeros(1, dtype=torch.int32, device="cuda"), want_lse=True)
    where["want_lse"] = True
    paged = dict(page_table=torch.arange(30, dtype=torch.int32, device="cuda")[None], want_lse=True)
    for f in (lambda c, w: K.attend_latent(q, c, R, cu, dev, lens_of([n]), n, 0.1, **w),
              lambda c, w: K.attend_latent_selected(q, c, R, ids, cu, dev, lens_of([n]), 0.1, **w)):
        ref = f(near, where)
        for got in (f(far, zero), f(far.unflatten(0, (30, 10)), paged)):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.gpu
def test_calls_of_two_threads_at_once():
    import threading
    jobs = []
    for seed, H in ((22, 16), (23, 64)):
        q, cache, where, _, args, ids, _, _ = run([1, 2], [3000, 700], H, 512, 64, 16, seed, 500)
        jobs.append(lambda stream=None, q=q, c=cache, w=where, a=args, i=ids: [
            *K.attend_latent(q, c, 512, *a, 3000, 0.04, want_lse=True, stream=stream, **w),
            *K.attend_latent_selected(q, c, 512, i, *a, 0.04, want_lse=True, stream=stream, **w)])
    alone = [job() for job in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(job, want):
        stream = torch.cuda.Stream()
        for _ in range(10):
            got = job(stream)
            stream.synchronize()
            wrong.extend(i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=pair) for pair in zip(jobs, alone)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# ---------------------------------------------------------------------------
# Refusals (no GPU)
# ---------------------------------------------------------------------------

AT = dict(q=1 << 32, cache=2 << 32, table=3 << 32, starts=4 << 32, lens=5 << 32, ids=6 << 32, cud=7 << 32, ws=8 << 32,
          o=9 << 32, lse=10 << 32)


def _call(selected=False, cu=(0, 1, 2), H=16, R=512, P=64, qs=None, cs=None, rows=1000, per_seq=10, page=16, paged=True,
          max_len=100, width=64, scale=0.1, nb=1 << 40, nseq=None, **at):
    at = {**AT, **at}
    p = lambda n: None if at[n] is None else ctypes.c_void_p(at[n])
    cu = np.asarray(cu, dtype=np.int32)
    nseq = len(cu) - 1 if nseq is None else nseq
    W = R + P
    keys = (p("q"), H * W if qs is None else qs, p("cache"), W if cs is None else cs, rows, p("table") if paged else None,
            per_seq, page, p("starts"), p("lens"))
    rest = (cu.ctypes.data_as(ctypes.c_void_p), p("cud"), nseq, H, R, P, scale, p("ws"), nb, p("o"), p("lse"), None)
    if selected:
        return K.lib().kpool_attend_latent_selected(*keys, p("ids"), width, *rest)
    return K.lib().kpool_attend_latent(*keys, max_len, *rest)


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(H=0), -1), (dict(H=65537), -2), (dict(R=0), -1), (dict(R=12), -1), (dict(R=520), -2), (dict(P=-8), -1),
    (dict(P=4), -1), (dict(P=72), -2), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(qs=16 * 576 - 8), -1), (dict(qs=16 * 576 + 4), -1), (dict(qs=(1 << 24) + 8), -1), (dict(cs=568), -1),
    (dict(cs=580), -1), (dict(cs=(1 << 24) + 8), -1), (dict(rows=-1), -1), (dict(rows=1 << 31), -1), (dict(page=0), -1),
    (dict(per_seq=-1), -1), (dict(per_seq=1 << 28, page=16), -1), (dict(q=None), -1), (dict(cache=None), -1),
    (dict(lens=None), -1), (dict(cud=None), -1), (dict(o=None), -1), (dict(paged=False, starts=None), -1),
    (dict(q=(1 << 32) + 2), -1), (dict(cache=(2 << 32) + 8), -1), (dict(o=(9 << 32) + 8), -1), (dict(ws=(8 << 32) + 4), -1),
    (dict(lens=(5 << 32) + 2), -1), (dict(table=(3 << 32) + 1), -1), (dict(cud=(7 << 32) + 2), -1),
    (dict(lse=(10 << 32) + 2), -1), (dict(ws=None), -3), (dict(nb=100), -3), (dict(cu=(0, 2, 1)), -1), (dict(cu=(1, 2)), -1),
    (dict(nseq=0), -1), (dict(cu=(0, 1 << 28)), -2)])
def test_refuses(selected, kw, code):
    assert _call(selected, **kw) == code


def test_refuses_lengths_and_lists():
    assert _call(max_len=-1) == -1 and _call(max_len=0x7FFFFF01) == -1
    assert _call(True, width=-1) == -1 and _call(True, width=(1 << 30) + 1) == -1 and _call(True, ids=None) == -1
    assert _call(True, ids=(6 << 32) + 2) == -1
    assert _call(cu=(0, 200000), max_len=0x7FFFFF00) == -2 and _call(True, cu=(0, 1 << 20), width=1 << 20) == -2
    assert _call(cu=(0, 0), q=None, o=None, lens=None, cud=None, ws=None) == 0


def test_refuses_products_past_64_bits():
    """Rows and list entries, each within its own bound, whose tiles a 64-bit product would wrap to few or negative."""
    cu = np.arange(65537, dtype=np.int64) * 32000
    assert _call(True, cu=cu, H=65536, R=8, P=0, width=1 << 30) == -2
    assert _call(cu=cu, H=65536, R=8, P=0, max_len=0x7FFFFF00) == -2


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("out", ["o", "lse", "ws"])
@pytest.mark.parametrize("over", ["q", "cache", "table", "starts", "lens", "cud", "ids", "lse", "ws", "o"])
def test_refuses_overlaps(selected, out, over):
    if out == over or (over == "ids" and not selected):
        return
    paged = over != "starts"
    assert _call(selected, paged=paged, **{out: AT[over]}) == -1
    assert b"overlaps" in K.lib().kpool_last_error()


def test_workspace_bytes():
    assert K.attend_latent_workspace_bytes([0, 1], 64, 16, 512, 64) == 0    # one tile: no parts
    one = K.attend_latent_workspace_bytes([0, 1], 640, 16, 512, 64)
    assert one == 10 * 32 + 2 * 10 * 16 * 513 * 4
    assert K.attend_latent_workspace_bytes([0, 1], 1 << 20, 16, 512, 64) == 256 * (32 + 2 * 16 * 513 * 4)
    assert K.attend_latent_selected_workspace_bytes(0, 2048, 16, 512, 64) <= one
    for bad in (lambda: K.attend_latent_workspace_bytes([0, 1], -1, 16, 512, 64),
                lambda: K.attend_latent_workspace_bytes([0, 1], 5, 16, 13, 64),
                lambda: K.attend_latent_selected_workspace_bytes(-1, 5, 16, 512, 64),
                lambda: K.attend_latent_selected_workspace_bytes(1, 5, 0, 512, 64)):
        with pytest.raises(K.KpoolError):
            bad()


@pytest.mark.gpu
def test_refuses_in_python():
    q, cache, where, _ = make([2], [40], 4, 64, 8, 16, 24)
    cu, dev = cu_of([2])
    lens = lens_of([40])
    call = lambda q=q, cache=cache, rank=64, lens=lens, **kw: K.attend_latent(q, cache, rank, cu, dev, lens, 40, 0.1,
                                                                              **{**where, **kw})
    call()
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (dict(rank=0), dict(rank=73), dict(q=q.float()), dict(cache=cache[..., :64]), dict(cache=cache.float()),
                dict(lens=lens.long()), dict(lens=lens_of([40, 1])), dict(page_table=None), dict(k_starts=start),
                dict(page_table=where["page_table"][0]), dict(cache=cache.flatten(0, 1)), dict(q=q[:1]),
                dict(cache=cache[:, :7]), dict(page_table=None, k_starts=start),
                dict(cache=torch.cat([cache, cache], 2)[..., ::2])):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError, match="autograd"):
        call(cache=cache.clone().requires_grad_())
