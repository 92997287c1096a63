"""Expanded latent attention in 64 bits: attend_reference's formulas and bounds with keys of D + P values,
the last P of which all heads share, and values of D.  The positional gradient sums the key heads' shares
(each by its own bound) in fp32, H u of their absolute sum on top."""
import math

import torch

from attend_reference import H, U, causal_counts, one_head, sequences

BF16 = torch.bfloat16


def make(cu_q, cu_k, Hq, Hkv, D, P, seed, pad=0, gain=2.0):
    """q, k, k_pe, v: k and v as the halves of one projection's heads, q and k_pe slices of wider rows (pad
    more values a token), with two more tokens of NaN behind the last sequence."""
    g = torch.Generator().manual_seed(seed)

    def rows(T, width, scale):
        wide = (scale * torch.randn(T + 2, width + pad, generator=g)).to(BF16).cuda()
        wide[T:] = float("nan")
        return wide[:, :width]
    q = rows(int(cu_q[-1]), Hq * (D + P), gain).unflatten(1, (Hq, D + P))
    kv = rows(int(cu_k[-1]), Hkv * 2 * D, 1.0).unflatten(1, (Hkv, 2 * D))
    return q, kv[:, :, :D], rows(int(cu_k[-1]), P, 1.0), kv[:, :, D:]


def full_keys(k, k_pe, c, d, g):
    return torch.cat([k[c:d, g], k_pe[c:d]], 1).double()


def check(q, k, k_pe, v, cu_q, cu_k, scale, o, lse):
    G = q.shape[1] // k.shape[1]
    for a, b, c, d in sequences(cu_q, cu_k):
        if a == b:
            continue
        if c == d:
            assert (o[a:b] == 0).all() and (lse[a:b] == -math.inf).all()
            continue
        count = causal_counts(b - a, d - c)
        for h in range(q.shape[1]):
            kk = full_keys(k, k_pe, c, d, h // G)
            ro, rl, _, to, tl = one_head(q[a:b, h].double(), kk, v[c:d, h // G].double(), count, scale)
            err = (o[a:b, h].double() - ro).abs()
            assert (err <= to).all(), (a, h, float((err - to).max()))
            got, empty = lse[a:b, h].double(), rl == -math.inf
            assert torch.equal(got == -math.inf, empty)
            assert ((got - rl).abs() <= tl)[~empty].all()
            assert (o[a:b, h][empty] == 0).all()


def check_backward(q, k, k_pe, v, d_o, o, lse, cu_q, cu_k, scale, dq, dk, dk_pe, dv):
    """attend_reference.check_backward's derivation, with the positional gradient."""
    Hkv, D = k.shape[1:]
    G, W = q.shape[1] // Hkv, q.shape[2]
    tiny = 2.0 ** -126
    for a, b, c, d in sequences(cu_q, cu_k):
        lq, lk = b - a, d - c
        if lk == 0:
            assert (dq[a:b] == 0).all()
            continue
        seen = (causal_counts(lq, lk) > 0).repeat_interleave(G, 0)
        pe_ref = torch.zeros(lk, W - D, dtype=torch.float64, device="cuda")
        pe_bound, pe_abs = pe_ref.clone(), pe_ref.clone()

        def near(got, ref, bound):
            tol = bound + H * (ref.abs() + bound) + tiny
            err = (got.double() - ref).abs()
            assert (err <= tol).all(), (a, float((err - tol).max()))

        for g in range(Hkv):
            hs = slice(g * G, g * G + G)
            rows = lambda t: t[a:b, hs].double().reshape(lq * G, t.shape[2])
            qq, oo, ee = rows(q), rows(o), rows(d_o)
            kk, vv = full_keys(k, k_pe, c, d, g), v[c:d, g].double()
            l64 = lse[a:b, hs].double().reshape(-1, 1)
            p = torch.where(seen, (scale * (qq @ kk.t()) - l64.clamp(min=-1e30)).exp(), 0.0)
            e = torch.where(seen, scale * (qq.abs() @ kk.abs().t()) * (W + 8) * U, 0.0).amax(1, keepdim=True) \
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
            bp = p * (H + ep + 2 * n) + tiny * seen
            bs = ds.abs() * (H + ep + 2 * n) + 2 * p * e2 + tiny * (1 + (dp - delta).abs()) * seen
            near(dv[c:d, g], p.t() @ ee, bp.t() @ ee.abs())
            near(rows(dq), scale * ds @ kk, scale * bs @ kk.abs())
            kref, kbound = scale * ds.t() @ qq, scale * bs.t() @ qq.abs()
            near(dk[c:d, g], kref[:, :D], kbound[:, :D])
            pe_ref += kref[:, D:]
            pe_bound += kbound[:, D:]
            pe_abs += kref[:, D:].abs()
        near(dk_pe[c:d], pe_ref, pe_bound + Hkv * U * (pe_abs + pe_bound))
