"""A latent attention layer over what its indexer selects: index queries and keys normalised, turned, pooled, scored,
selected and expanded by Selector.run, the attention's queries and cache rows turned, and attend_latent_selected over
the token ids that the selection gave.

The selection is checked by its oracle on what rotary itself gives, the attention against 64 bits over the ids
(tolerances: latent_reference.py)."""
import numpy as np
import pytest
import torch

import oracle
from attend_reference import cu_of
from gpu_helpers import check_selection_vs_oracle
from latent_reference import BF16, check, lens_of
from pool_score_top_amd import kpool as K
from pool_score_top_amd import synth

H, R, P = 16, 64, 32


def select(cu, kpool, budget, tail, q_lo, q_hi, seed):
    """The selector, its ids, and what the oracle selects from."""
    T = cu[-1]
    r = synth.host_inputs(synth.workload("sq4096", T=T, kpool=kpool, budget=budget), seed)
    dev = {n: torch.from_numpy(r[n].view(np.int16) if r[n].dtype == np.uint16 else r[n]).cuda() for n in ("q", "k", "w")}
    g = torch.Generator().manual_seed(seed)
    norm = ((1 + 0.2 * torch.randn(128, generator=g)).cuda(), torch.randn(128, generator=g).cuda(), 1e-6)
    freqs, factor = K.rotary_frequencies(32, scale=40.0, trained=4096)
    sel = K.Selector(cu, kpool, budget, 32, 128, tail=tail, q_lo=q_lo, q_hi=q_hi, rotary=(freqs, 0, False, factor))
    out = sel.run(dev["q"], dev["k"], dev["w"], k_norm=norm)
    turn = lambda x: K.rotary(x, sel.positions, freqs, factor=factor)
    bits = [t.cpu().numpy().view(np.uint16) for t in (turn(dev["q"]), turn(K.layer_norm(dev["k"], *norm)[0]))]
    ref = oracle.select(*bits, r["w"], np.asarray(cu, np.int32), kpool, budget, tail=tail)
    cu_pools, _ = oracle.count_pools(cu, kpool, tail=tail)
    seq, t = oracle.row_positions(np.arange(T), cu)
    nvis = oracle.visible_pools(t, kpool, cu_pools[seq + 1] - cu_pools[seq])
    rows = slice(sel.q_lo, sel.q_hi)
    scores = ref["scores"][rows]
    check_selection_vs_oracle(out["pool_ids"].cpu().numpy(), scores, nvis[rows], budget, "latent layer")
    return sel, out["token_ids"]


def attention(cu, positions, seed, page):
    """The attention's own queries and cache rows, positions on their last P values, and where the cache's rows are:
    each sequence's rows as they lie in memory."""
    T = cu[-1]
    g = torch.Generator().manual_seed(seed)
    freqs, factor = K.rotary_frequencies(P // 2, scale=40.0, trained=4096)
    how = dict(begin=R, interleaved=True, factor=factor)
    q = torch.randn(T, H, R + P, generator=g).to(BF16).cuda()
    c = torch.randn(T, R + P, generator=g).to(BF16).cuda()
    for x in (q, c):
        K.rotary(x, positions, freqs, out=x, **how)
    rows = [c[a:b] for a, b in zip(cu[:-1], cu[1:])]
    if not page:
        return q, c, dict(k_starts=torch.tensor(cu[:-1], dtype=torch.int32, device="cuda")), rows
    per = [-(-len(x) // page) for x in rows]
    cache = torch.full((sum(per) + 1, page, R + P), float("nan"), dtype=BF16, device="cuda")
    order = torch.randperm(sum(per) + 1, generator=g)
    table = torch.full((len(rows), max(per)), -1, dtype=torch.int32)
    at = 0
    for s, x in enumerate(rows):
        table[s, :per[s]] = order[at:at + per[s]].to(torch.int32)
        at += per[s]
        for i in range(per[s]):
            part = x[i * page:(i + 1) * page]
            cache[int(table[s, i]), :len(part)] = part
    return q, cache, dict(page_table=table.cuda()), rows


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("cu,kpool,budget,tail,q_lo,q_hi", [
    ([0, 700, 701, 701, 1500], 4, 64, False, 0, None), ([0, 700, 701, 701, 1500], 4, 64, True, 0, None),
    ([0, 1003], 1, 200, False, 0, None), ([0, 300, 1200], 5, 7, True, 0, None), ([0, 90, 400], 4, 128, False, 0, None),
    ([0, 300, 1000, 1500], 4, 32, False, 200, 1100), ([0, 300, 1000, 1500], 4, 32, True, 650, 651)])
def test_prompts_over_what_they_select(cu, kpool, budget, tail, q_lo, q_hi, page):
    """Every row of a range over its own list: sequences cut by the range, empty ones, lists wider than the tokens."""
    sel, ids = select(cu, kpool, budget, tail, q_lo, q_hi, 3)
    q, cache, where, rows = attention(cu, sel.positions, 4, page)
    (cu_q, cu_k), (cqd, _) = sel.attend_cu, sel.attend_cu_dev
    k_lens = np.diff(cu_k).tolist()
    mine = q[sel.q_lo:sel.q_hi]
    o, lse = K.attend_latent_selected(mine, cache, R, ids, cu_q, cqd, lens_of(k_lens), 0.1, want_lse=True, **where)
    check(mine, [x[:n] for x, n in zip(rows, k_lens)], np.diff(cu_q).tolist(), k_lens, R, 0.1, o, lse, ids)
    if sel.max_pools > sel.budget:
        return
    # everything visible is selected: the whole form obeys the same bounds
    whole = K.attend_latent(mine, cache, R, cu_q, cqd, lens_of(k_lens), max(k_lens), 0.1, want_lse=True, **where)
    check(mine, [x[:n] for x, n in zip(rows, k_lens)], np.diff(cu_q).tolist(), k_lens, R, 0.1, *whole, ids)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 64])
def test_new_tokens_over_what_they_select(page):
    """A serving step: the last row of each sequence over its list."""
    cu, kpool, budget = [0, 700, 701, 1203, 1500], 4, 32
    sel, ids = select(cu, kpool, budget, False, 0, None, 5)
    q, cache, where, rows = attention(cu, sel.positions, 6, page)
    k_lens = np.diff(cu).tolist()
    last = torch.tensor(cu[1:], device="cuda") - 1
    q1, ids1 = q[last], ids[last]
    cu1, dev1 = cu_of([1] * len(k_lens))
    o, lse = K.attend_latent_selected(q1, cache, R, ids1, cu1, dev1, lens_of(k_lens), 0.1, want_lse=True, **where)
    check(q1, rows, [1] * len(k_lens), k_lens, R, 0.1, o, lse, ids1)
