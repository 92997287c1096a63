"""Attention and its gradients in 64 bits, one sequence and head at a time, with the bounds
that the kernels' arithmetic obeys.

u = 2^-24 is fp32's half step, h = 2^-8 bf16's.  A score is a sum of D exact products in fp32
(relative (D + 8) u of sum |q k|, the scaling and the hardware's 2^x included); call the largest
such error of a row e.  A weight p is then off by 2 e relative and is rounded to bf16 (h) for
its product with v; sums over n keys in fp32, in whatever order, are off by n u of their terms.
So with A = sum p |v|:
   |o - o64| <= (h + 4 e + 3 n u) A, and h |o| for the output's rounding
   |lse - lse64| <= 2 e + 2 n u + 4 u |lse|
"""
import math

import torch

U, H = 2.0 ** -24, 2.0 ** -8


def sequences(cu_q, cu_k):
    for s in range(len(cu_q) - 1):
        yield int(cu_q[s]), int(cu_q[s + 1]), int(cu_k[s]), int(cu_k[s + 1])


def causal_counts(lq, lk):
    """[lq, lk]: how often a row counts a key (once, up to its position)."""
    t = torch.arange(lk - lq, lk, device="cuda")
    return (torch.arange(lk, device="cuda") <= t[:, None]).double()


def list_counts(ids, lk):
    """[lq, lk]: how often a row's list names a key it sees."""
    lq = ids.shape[0]
    t = torch.arange(lk - lq, lk, device="cuda")[:, None]
    ok = (ids >= 0) & (ids <= t)
    n = torch.zeros(lq, lk + 1, dtype=torch.float64, device="cuda")
    n.scatter_add_(1, torch.where(ok, ids, lk).long(), ok.double())
    return n[:, :lk]


def one_head(q, k, v, count, scale):
    """q [lq, D], k, v [lk, D] in 64 bits, count [lq, lk]: (o, lse, p, tol_o, tol_lse)."""
    lq, D = q.shape
    lk = k.shape[0]
    if lk == 0:
        z = torch.zeros(lq, D, dtype=torch.float64, device=q.device)
        return z, torch.full((lq,), -math.inf, dtype=torch.float64, device=q.device), None, z, z[:, 0]
    seen = count > 0
    s = torch.where(seen, scale * (q @ k.t()) + count.clamp(min=1).log(), -math.inf)
    lse = torch.logsumexp(s, 1)
    p = torch.where(seen, (s - lse.clamp(min=-1e30)[:, None]).exp(), 0.0)
    vz = torch.where(seen.any(0)[:, None], v, 0.0)
    o = p @ vz
    e = torch.where(seen, scale * (q.abs() @ k.abs().t()), 0.0).amax(1) * (D + 8) * U
    n = count.sum(1)
    A = p @ vz.abs()
    tol = (H + 4 * e + 3 * (n + 64) * U)[:, None] * A
    tol = tol + H * (o.abs() + tol)
    return o, lse, p, tol, 2 * e + 2 * (n + 64) * U + 4 * U * lse.abs().clamp(max=1e30)


def check(q, k, v, cu_q, cu_k, scale, o, lse, ids=None):
    """Every sequence and head of o (and lse, where given) against 64 bits."""
    G = q.shape[1] // k.shape[1]
    for a, b, c, d in sequences(cu_q, cu_k):
        if a == b:
            continue
        count = causal_counts(b - a, d - c) if ids is None else list_counts(ids[a:b], d - c)
        for h in range(q.shape[1]):
            kk, vv = k[c:d, h // G].double(), v[c:d, h // G].double()
            # (what no row of the sequence sees has no part in it, NaN or not)
            keep = (count > 0).any(0)[:, None]
            kk, vv = torch.where(keep, kk, 0.0), torch.where(keep, vv, 0.0)
            ro, rl, _, to, tl = one_head(q[a:b, h].double(), kk, vv, count, scale)
            err = (o[a:b, h].double() - ro).abs()
            assert (err <= to).all(), (a, h, float((err - to).max()))
            if lse is not None:
                got = lse[a:b, h].double()
                empty = rl == -math.inf
                assert torch.equal(got == -math.inf, empty)
                assert ((got - rl).abs() <= tl)[~empty].all()
                assert (o[a:b, h][empty] == 0).all()


def make(cu_q, cu_k, Hq, Hkv, D, seed, pad=0, gain=2.0):
    """bf16 q, k, v as slices of wider rows (pad more values per token) with two more tokens of
    NaN behind the last sequence."""
    g = torch.Generator().manual_seed(seed)

    def rows(T, heads, scale):
        wide = (scale * torch.randn(T + 2, heads * D + pad, generator=g)).to(torch.bfloat16).cuda()
        wide[T:] = float("nan")
        return wide[:, :heads * D].unflatten(1, (heads, D))
    return rows(int(cu_q[-1]), Hq, gain), rows(int(cu_k[-1]), Hkv, 1.0), rows(int(cu_k[-1]), Hkv, 1.0)


def cu_of(lens):
    import numpy as np
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return cu, torch.from_numpy(cu).cuda()


def check_backward(q, k, v, d_o, o, lse, cu_q, cu_k, scale, dq, dk, dv):
    """The gradients of every sequence and key head against the formulas in 64 bits with the
    given lse (as the backward pass has it).

    P = exp(s - lse) has the relative error ep = 4 e + 16 u (1 + |lse|); dP is a sum of D
    products (D + 8) u; delta = sum P dP may be taken as sum do o with the forward pass's o,
    which is off by (h + 4 e + 3 n u) sum p |v| and h |o| (see above); dS = P (dP - delta)
    carries these and is rounded to bf16 (h) for its products, as P is; sums over n rows or
    keys add n u, the outputs' rounding h.

    Below 2^-126, the smallest normal number of fp32 and bf16, the hardware's 2^x and the
    matrix products give 0 (no subnormals), whatever the relative bounds say: P, dS and each
    output are off by up to that much on top, P's part reaching dS through |dP - delta|."""
    G = q.shape[1] // k.shape[1]
    D = q.shape[2]
    for a, b, c, d in sequences(cu_q, cu_k):
        lq, lk = b - a, d - c
        if lk == 0:
            assert (dq[a:b] == 0).all()
            continue
        seen = (causal_counts(lq, lk) > 0).repeat_interleave(G, 0)
        for g in range(k.shape[1]):
            hs = slice(g * G, g * G + G)
            rows = lambda t: t[a:b, hs].double().reshape(lq * G, D)
            qq, oo, ee = rows(q), rows(o), rows(d_o)
            kk, vv = k[c:d, g].double(), v[c:d, g].double()
            l64 = lse[a:b, hs].double().reshape(-1, 1)
            p = torch.where(seen, (scale * (qq @ kk.t()) - l64.clamp(min=-1e30)).exp(), 0.0)
            e = torch.where(seen, scale * (qq.abs() @ kk.abs().t()) * (D + 8) * U, 0.0).amax(1, keepdim=True) \
                if lq else p.sum(1, keepdim=True)
            ep = 4 * e + 16 * U * (1 + l64.abs().clamp(max=1e30) * (l64 > -math.inf))
            dp = ee @ vv.t()
            delta = (p * dp).sum(1, keepdim=True)
            ds = p * (dp - delta)
            n = (lq * G + lk + 64) * U
            o_off = (H + 4 * e + 3 * n) * (p @ vv.abs())
            o_off = o_off + H * ((p @ vv).abs() + o_off)
            e2 = (D + 8) * U * (ee.abs() @ vv.abs().t() + (ee * oo).abs().sum(1, keepdim=True))
            e2 = e2 + (ee.abs() * o_off).sum(1, keepdim=True)
            tiny = 2.0 ** -126
            bp = p * (H + ep + 2 * n) + tiny * seen
            bs = ds.abs() * (H + ep + 2 * n) + 2 * p * e2 + tiny * (1 + (dp - delta).abs()) * seen
            for got, ref, bound in (
                    (dv[c:d, g].double(), p.t() @ ee, bp.t() @ ee.abs()),
                    (dk[c:d, g].double(), scale * ds.t() @ qq, scale * bs.t() @ qq.abs()),
                    (rows(dq), scale * ds @ kk, scale * bs @ kk.abs())):
                tol = bound + H * (ref.abs() + bound) + tiny
                err = (got - ref).abs()
                assert (err <= tol).all(), (a, g, float((err - tol).max()))
