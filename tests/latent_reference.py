"""Latent attention over a cache in 64 bits, by the bounds of attend_reference.one_head: a score is a
sum of R + P products, the value of a token its row's first R values."""
import math

import numpy as np
import torch

from attend_reference import causal_counts, cu_of, list_counts, one_head

BF16 = torch.bfloat16


def make(q_lens, k_lens, H, R, P, page, seed, gain=1.0, pad=0, spare=3):
    """q, cache, how the cache is addressed (keyword arguments) and each sequence's rows as they lie in
    memory.  Rows of no token hold NaN, those behind a sequence's tokens in its last page among them."""
    g = torch.Generator().manual_seed(seed)
    Tq, W = sum(q_lens), R + P

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    q = (gain * normal(Tq + 2, H * W + pad)).to(BF16).cuda()
    q[Tq:] = float("nan")
    q = q[:, :H * W].unflatten(1, (H, W))
    rows = [normal(n, W).to(BF16).cuda() for n in k_lens]
    if page:
        per = [-(-n // page) for n in k_lens]
        total = sum(per) + spare
        wide = torch.full((total * page, W + pad), float("nan"), dtype=BF16, device="cuda")
        order = torch.randperm(total, generator=g)
        table = torch.full((len(k_lens), max(per + [1]) + 2), -7, dtype=torch.int32)
        at = 0
        for s, n in enumerate(per):
            table[s, :n] = order[at:at + n].to(torch.int32)
            at += n
            t = torch.arange(k_lens[s])
            wide[(table[s].long()[t // page] * page + t % page).cuda(), :W] = rows[s]
        return q, wide[:, :W].unflatten(0, (total, page)), dict(page_table=table.cuda()), rows
    order = torch.randperm(len(k_lens), generator=g).tolist()
    wide = torch.full((sum(k_lens) + spare + 2 * len(k_lens), W + pad), float("nan"), dtype=BF16, device="cuda")
    starts, at = [0] * len(k_lens), 1
    for s in order:
        starts[s] = at
        wide[at:at + k_lens[s], :W] = rows[s]
        at += k_lens[s] + 2
    return q, wide[:, :W], dict(k_starts=torch.tensor(starts, dtype=torch.int32, device="cuda")), rows


def check(q, rows, q_lens, k_lens, R, scale, o, lse, ids=None, there=None):
    """Every sequence and head of o and lse against 64 bits; there[s]: which tokens the cache holds."""
    at = 0
    for s, (lq, lk) in enumerate(zip(q_lens, k_lens)):
        a, at = at, at + lq
        if lq == 0:
            continue
        if lk == 0:
            assert (o[a:at] == 0).all() and (lse[a:at] == -math.inf).all()
            continue
        count = causal_counts(lq, lk) if ids is None else list_counts(ids[a:at], lk)
        if there is not None:
            count = count * there[s].double()
        c = torch.where((count > 0).any(0)[:, None], rows[s].double(), 0.0)
        for h in range(q.shape[1]):
            ro, rl, _, to, tl = one_head(q[a:at, h].double(), c, c[:, :R], count, scale)
            err = (o[a:at, h].double() - ro).abs()
            assert (err <= to).all(), (s, h, float((err - to).max()))
            got, empty = lse[a:at, h].double(), rl == -math.inf
            assert torch.equal(got == -math.inf, empty)
            assert ((got - rl).abs() <= tl)[~empty].all()
            assert (o[a:at, h][empty] == 0).all()


def lens_of(k_lens):
    return torch.tensor(k_lens, dtype=torch.int32, device="cuda")


def lists(q_lens, k_lens, width, seed, kind):
    """Token ids: distinct ones and -1 in any places ("holes"), all -1 ("none"), any numbers, repeated
    and out of range among them ("wild"), or what each row sees in order ("all")."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for lq, lk in zip(q_lens, k_lens):
        t = torch.arange(lk - lq, lk)[:, None]
        if kind == "none":
            ids = torch.full((lq, width), -1)
        elif kind == "all":
            ids = torch.arange(width).expand(lq, width)
            ids = torch.where(ids <= t, ids, -1)
        elif kind == "wild":
            ids = torch.randint(-5, max(lk, 1) + 5, (lq, width), generator=g)
        else:
            n = max(lk, width)
            ids = torch.stack([torch.randperm(n, generator=g)[:width] for _ in range(lq)]) if lq else torch.zeros(0, width)
            ids = torch.where(ids <= t, ids, -1)
        out.append(ids)
    return torch.cat(out).to(torch.int32).cuda()
