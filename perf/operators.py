"""Cases and plain forms of the attention layer's operators around the selection.

Four paths of one sparse-attention layer, as a program that uses the selection runs them:

  attend    attention of query rows over all the keys they see (packed sequences, grouped
            heads, queries at the end of their sequence's keys), forward
  train     the same attention with its backward pass: one training step
  selected  attention of query rows over the token ids that the selection gave them
  norm      layer norm of index keys or hidden states, forward, or forward and backward
            with the weight's and bias's gradients

`own` is False for the plain forms (elementary torch operations in fp32, rounded once at
the end) and True for the library's kernels.
"""
import math

import torch

own = False

_BF16 = torch.bfloat16


def listed():
    return [
        # a long document read in one pass (prefill), grouped heads
        {"name": "prompt_long", "kind": "attend", "q_lens": "16384", "k_lens": "16384",
         "hq": 16, "hkv": 2, "d": 128},
        # a prefill batch of requests of very different lengths, one of a single token
        {"name": "prompt_packed", "kind": "attend", "q_lens": "4097,2050,1500,513,33,1",
         "k_lens": "4097,2050,1500,513,33,1", "hq": 32, "hkv": 4, "d": 128},
        # one serving step: a batch of requests, one new token each, ragged long caches
        {"name": "tokens_batch", "kind": "attend", "q_lens": "1,1,1,1,1,1,1,1",
         "k_lens": "32768,30011,16385,9000,4096,1023,130,1", "hq": 32, "hkv": 4, "d": 128},
        # one new token of one short request: the smallest call, where latency counts
        {"name": "token_one", "kind": "attend", "q_lens": "1", "k_lens": "517", "hq": 8, "hkv": 8,
         "d": 64},
        # a training step over packed documents, grouped heads
        {"name": "train_packed", "kind": "train", "q_lens": "4096,2777,1000,319",
         "k_lens": "4096,2777,1000,319", "hq": 16, "hkv": 4, "d": 128},
        # a training step with one key head shared by all query heads and a narrow head
        {"name": "train_shared", "kind": "train", "q_lens": "2048", "k_lens": "2048", "hq": 8,
         "hkv": 1, "d": 64},
        # the last rows of a 64k-token prompt over the 2048 tokens (512 pools of 4) each selected
        {"name": "selected_rows", "kind": "selected", "q_lens": "2048", "k_lens": "65536",
         "hq": 32, "hkv": 2, "d": 128, "kpool": 4, "budget": 512},
        # one serving step over selected tokens: one new token per request
        {"name": "selected_tokens", "kind": "selected", "q_lens": "1,1,1,1,1,1,1,1",
         "k_lens": "65536,50001,32768,20000,10007,4096,900,1", "hq": 32, "hkv": 2, "d": 128,
         "kpool": 4, "budget": 512},
        # index keys of a 512k-token sequence normalised before they are pooled
        {"name": "norm_keys", "kind": "norm", "rows": 524288, "n": 128, "type": "bf16", "pad": 0,
         "backward": False},
        # one new token's index key: the smallest call
        {"name": "norm_token", "kind": "norm", "rows": 1, "n": 128, "type": "bf16", "pad": 0,
         "backward": False},
        # a training step of the norm over hidden states
        {"name": "norm_train", "kind": "norm", "rows": 8192, "n": 4096, "type": "bf16", "pad": 0,
         "backward": True},
        # a training step in fp32 over an odd width, a slice of a wider projection
        {"name": "norm_odd", "kind": "norm", "rows": 5003, "n": 1237, "type": "f32", "pad": 91,
         "backward": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 7, 8, 16])
    return hkv * g, hkv


def draw(rng):
    kind = rng.choice(["attend", "attend", "train", "selected", "norm"])
    if kind == "norm":
        n = _log_int(rng, 16, 8192)
        most = 33_554_432 // n
        backward = rng.random() < 0.6
        return {"kind": "norm", "rows": _log_int(rng, 1, min(most, 524288)), "n": n,
                "type": rng.choice(["bf16", "f32"]), "pad": rng.choice([0, 0, 8, 37]),
                "backward": backward}
    hq, hkv = _heads(rng)
    if kind == "selected":
        nseq = rng.randint(1, 6)
        rows = [_log_int(rng, 1, 300) for _ in range(nseq)]
        kpool = rng.choice([1, 2, 4, 5])
        return {"kind": "selected", "q_lens": ",".join(map(str, rows)),
                "k_lens": ",".join(str(n + _log_int(rng, 1, 20000)) for n in rows), "hq": hq,
                "hkv": hkv if hkv < 8 else 2 if hq % 2 == 0 else 1, "d": rng.choice([64, 128]),
                "kpool": kpool, "budget": _log_int(rng, 1, 2048 // kpool)}
    d = rng.choice([64, 80, 128])
    if kind == "train":
        lens = [_log_int(rng, 1, 2600) for _ in range(rng.randint(1, 4))]
        text = ",".join(map(str, lens))
        return {"kind": "train", "q_lens": text, "k_lens": text, "hq": min(hq, 16 // hkv * hkv),
                "hkv": hkv, "d": d}
    nseq = rng.randint(1, 6)
    form = rng.choice(["prompt", "rows", "token"])
    if form == "prompt":
        q = [_log_int(rng, 1, 4000) for _ in range(nseq)]
        k = list(q)
        hq = min(hq, 32 // hkv * hkv)
    elif form == "rows":
        q = [_log_int(rng, 1, 500) for _ in range(nseq)]
        k = [n + _log_int(rng, 1, 10000) for n in q]
        hq = min(hq, 32 // hkv * hkv)
    else:
        q = [1] * nseq
        k = [_log_int(rng, 1, 60000) for _ in q]
    return {"kind": "attend", "q_lens": ",".join(map(str, q)), "k_lens": ",".join(map(str, k)),
            "hq": hq, "hkv": hkv, "d": d}


def _lens(text):
    return [int(x) for x in text.split(",")]


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def work(case):
    if case["kind"] == "norm":
        rows, n = case["rows"], case["n"]
        size = 2 if case["type"] == "bf16" else 4
        if not case["backward"]:
            return {"bytes": 2 * rows * n * size + 8 * n, "flops": 8 * rows * n}
        return {"bytes": 4 * rows * n * size + 8 * rows + 16 * n, "flops": 21 * rows * n}
    q, k = _lens(case["q_lens"]), _lens(case["k_lens"])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    tq, tk = sum(q), sum(k)
    rows = tq * hq * d * 2
    keys = tk * hkv * d * 2
    if case["kind"] == "selected":
        width = case["kpool"] * case["budget"]
        pairs = sum(min(width, b - a + i + 1) for a, b in zip(q, k) for i in range(a))
        read = sum(min(b, width * a) for a, b in zip(q, k)) * hkv * d * 2
        return {"bytes": 2 * rows + 2 * read + 4 * tq * width + 4 * tq * hq,
                "flops": 4 * d * hq * pairs}
    pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(q, k))
    if case["kind"] == "attend":
        return {"bytes": 2 * rows + 2 * keys + 4 * tq * hq, "flops": 4 * d * hq * pairs}
    return {"bytes": 4 * rows + 4 * keys + 4 * tq * hq, "flops": 14 * d * hq * pairs}


def _pool_ids(gen, q, k, kpool, budget):
    """Token ids as the selection gives them: distinct visible pools per row in random order,
    expanded to tokens, -1 past the row's tokens and where the pools run out."""
    out = []
    for lq, lk in zip(q, k):
        t = torch.arange(lk - lq, lk, device="cuda")
        npool = (lk + kpool - 1) // kpool
        score = torch.rand(lq, npool, device="cuda", generator=gen)
        score.masked_fill_(torch.arange(npool, device="cuda") > (t // kpool)[:, None], -1.0)
        top = score.topk(min(budget, npool), dim=1)
        pools = torch.where(top.values >= 0, top.indices, -1)
        ids = torch.full((lq, budget, kpool), -1, dtype=torch.int64, device="cuda")
        tok = pools[:, :, None] * kpool + torch.arange(kpool, device="cuda")
        ids[:, :pools.shape[1]] = torch.where((pools[:, :, None] >= 0) & (tok <= t[:, None, None]), tok, -1)
        out.append(ids.reshape(lq, budget * kpool))
    return torch.cat(out).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if case["kind"] == "norm":
        rows, n, pad = case["rows"], case["n"], case["pad"]
        dtype = _BF16 if case["type"] == "bf16" else torch.float32
        # (a projection's output: rows of different scale and offset)
        x = normal(rows, n + pad) * (0.5 + torch.rand(rows, 1, device="cuda", generator=gen)) + normal(rows, 1)
        st = {"case": case, "x": x.to(dtype)[:, :n], "eps": 1e-6,
              "weight": 1.0 + 0.2 * normal(n), "bias": 0.2 * normal(n)}
        if case["backward"]:
            st["dy"] = normal(rows, n).to(dtype)
        return st
    import numpy as np
    q, k = _lens(case["q_lens"]), _lens(case["k_lens"])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    st = {"case": case, "scale": 1.0 / math.sqrt(d), "q_max": max(q), "k_max": max(k),
          "cu_q": np.array(_cu(q), dtype=np.int32), "cu_k": np.array(_cu(k), dtype=np.int32),
          # (queries a little longer than the keys, so that some scores stand out)
          "q": (2.0 * normal(sum(q), hq, d)).to(_BF16), "k": normal(sum(k), hkv, d).to(_BF16),
          "v": normal(sum(k), hkv, d).to(_BF16)}
    st["cu_q_dev"] = torch.from_numpy(st["cu_q"]).cuda()
    st["cu_k_dev"] = torch.from_numpy(st["cu_k"]).cuda()
    if case["kind"] == "train":
        st["d_o"] = normal(sum(q), hq, d).to(_BF16)
    if case["kind"] == "selected":
        st["token_ids"] = _pool_ids(gen, q, k, case["kpool"], case["budget"])
    return st


def _norm(st):
    x = st["x"].float()
    mean = x.mean(dim=1)
    xc = x - mean[:, None]
    rstd = 1.0 / ((xc * xc).mean(dim=1) + st["eps"]).sqrt()
    xhat = xc * rstd[:, None]
    y = (xhat * st["weight"] + st["bias"]).to(st["x"].dtype)
    if not st["case"]["backward"]:
        return {"y": y}
    dy = st["dy"].float()
    wdy = dy * st["weight"]
    c1 = (wdy * xhat).mean(dim=1, keepdim=True)
    c2 = wdy.mean(dim=1, keepdim=True)
    dx = (rstd[:, None] * (wdy - c2 - xhat * c1)).to(st["x"].dtype)
    return {"y": y, "dx": dx, "dweight": (dy * xhat).sum(dim=0), "dbias": dy.sum(dim=0)}


def _padded(cu, longest):
    """Row numbers of the packed sequences as [nseq, longest], and which of them exist."""
    at = torch.arange(longest, device=cu.device)
    there = at < (cu[1:] - cu[:-1])[:, None]
    return torch.where(there, cu[:-1, None] + at, 0), there


def _attend(st):
    """Attention over whole keys, and its gradients where the state holds d_o."""
    case, scale = st["case"], st["scale"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    cu_q, cu_k = st["cu_q_dev"].long(), st["cu_k_dev"].long()
    qi, q_there = _padded(cu_q, st["q_max"])
    ki, k_there = _padded(cu_k, st["k_max"])
    nseq, lq, lk = qi.shape[0], st["q_max"], st["k_max"]

    def by_group(x):   # [T, hq, d] -> [nseq, hkv, lq * g, d]
        x = x[qi].float().view(nseq, lq, hkv, g, d)
        return x.permute(0, 2, 1, 3, 4).reshape(nseq, hkv, lq * g, d)

    def packed(x):     # and back, the rows that exist
        return x.view(nseq, hkv, lq, g, -1).permute(0, 2, 1, 3, 4).reshape(nseq, lq, hq, -1)[q_there]

    q = by_group(st["q"])
    k = st["k"][ki].float().permute(0, 2, 1, 3).contiguous()
    v = st["v"][ki].float().permute(0, 2, 1, 3).contiguous()
    t = torch.arange(lq, device=q.device) + (cu_k[1:] - cu_k[:-1] - cu_q[1:] + cu_q[:-1])[:, None]
    seen = (torch.arange(lk, device=q.device) <= t[:, :, None]) & k_there[:, None] & q_there[:, :, None]
    seen = seen[:, None, :, None].expand(nseq, 1, lq, g, lk).reshape(nseq, 1, lq * g, lk)
    s = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(scale).masked_fill_(~seen, -math.inf)
    m = s.amax(dim=3, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = s.sub_(m).exp_()
    total = p.sum(dim=3, keepdim=True)
    lse = packed(m + total.log()).squeeze(2)
    p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    o = packed(torch.matmul(p, v)).to(_BF16)
    if "d_o" not in st:
        return {"o": o, "lse": lse}
    d_o = by_group(st["d_o"])
    dp = torch.matmul(d_o, v.transpose(2, 3).contiguous())
    ds = p * (dp - (p * dp).sum(dim=3, keepdim=True)) * scale
    dq = packed(torch.matmul(ds, k)).to(_BF16)
    # (rows of absent queries have p = 0 and count for nothing here)
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), q).permute(0, 2, 1, 3)[k_there].to(_BF16)
    dv = torch.matmul(p.transpose(2, 3).contiguous(), d_o).permute(0, 2, 1, 3)[k_there].to(_BF16)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _selected(st):
    case = st["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    ids = st["token_ids"].long()
    rows = ids.shape[0]
    at = torch.arange(rows, device=ids.device)
    seq = (at[:, None] >= st["cu_q_dev"][1:]).sum(dim=1)
    flat = st["cu_k_dev"].long()[seq][:, None] + ids.clamp(min=0)
    k = st["k"][flat].float().permute(0, 2, 3, 1).contiguous()
    v = st["v"][flat].float().permute(0, 2, 1, 3).contiguous()
    q = st["q"].float().view(rows, hkv, g, d)
    s = torch.matmul(q, k).mul_(st["scale"]).masked_fill_((ids < 0)[:, None, None], -math.inf)
    m = s.amax(dim=3, keepdim=True)
    p = (s - m).exp()
    total = p.sum(dim=3, keepdim=True)
    o = torch.matmul(p / total, v).view(rows, hq, d).to(_BF16)
    return {"o": o, "lse": (m + total.log()).view(rows, hq)}


def run(state):
    kind = state["case"]["kind"]
    if not own:
        if kind == "norm":
            return _norm(state)
        return _selected(state) if kind == "selected" else _attend(state)
    from pool_score_top_amd import kpool as K
    st = state
    if kind == "norm":
        y, mean, rstd = K.layer_norm(st["x"], st["weight"], st["bias"], st["eps"],
                                     want_stats=st["case"]["backward"])
        if not st["case"]["backward"]:
            return {"y": y}
        dx, dw, db = K.layer_norm_backward(st["dy"], st["x"], st["weight"], mean, rstd)
        return {"y": y, "dx": dx, "dweight": dw, "dbias": db}
    cu = (st["cu_q"], st["cu_q_dev"], st["cu_k"], st["cu_k_dev"])
    if kind == "selected":
        o, lse = K.attend_selected(st["q"], st["k"], st["v"], st["token_ids"], *cu,
                                   scale=st["scale"], want_lse=True)
        return {"o": o, "lse": lse}
    o, lse = K.attend(st["q"], st["k"], st["v"], *cu, scale=st["scale"], want_lse=True)
    if kind == "attend":
        return {"o": o, "lse": lse}
    dq, dk, dv = K.attend_backward(st["d_o"], st["q"], st["k"], st["v"], o, lse, *cu,
                                   scale=st["scale"])
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _exact_norm(st):
    x, w = st["x"].double(), st["weight"].double()
    var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
    sd = (var + st["eps"]).sqrt()
    z = (x - mean) / sd
    out = {"y": torch.addcmul(st["bias"].double(), z, w)}
    if st["case"]["backward"]:
        dy = st["dy"].double()
        n = x.shape[1]
        dz = dy * w
        # the Jacobian of z: (I - 1 1^T / n - z z^T / n) / sd
        out["dx"] = (dz - (dz.sum(1, keepdim=True) + z * (dz * z).sum(1, keepdim=True)) / n) / sd
        out["dweight"] = torch.einsum("rn,rn->n", dy, z)
        out["dbias"] = dy.sum(0)
    return out


def _exact_rows(q, k, v, scale, seen, d_o=None):
    """One sequence and one key head in 64 bits: q [rows, g, d], k and v [keys, d], seen
    [rows, keys]; the keys' weights come from log_softmax."""
    rows, g, d = q.shape
    s = (q.reshape(rows * g, d) @ k.t() * scale).view(rows, g, -1)
    s = s.masked_fill(~seen[:, None], -math.inf)
    lse = torch.logsumexp(s, dim=2)
    w = torch.exp(s - lse[:, :, None]).view(rows * g, -1)
    o = w @ v
    if d_o is None:
        return o.view(rows, g, d), lse
    e = d_o.reshape(rows * g, d)
    dw = e @ v.t()
    dsc = scale * (w * dw - w * (e * o).sum(1, keepdim=True))
    return (o.view(rows, g, d), lse, (dsc @ k).view(rows, g, d), dsc.t() @ q.reshape(rows * g, d),
            w.t() @ e)


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "norm":
        return _exact_norm(st)
    q_lens, k_lens = _lens(case["q_lens"]), _lens(case["k_lens"])
    g, hkv = case["hq"] // case["hkv"], case["hkv"]
    names = ["o", "lse", "dq", "dk", "dv"] if case["kind"] == "train" else ["o", "lse"]
    parts = {n: [] for n in names}
    for i, (lq, lk) in enumerate(zip(q_lens, k_lens)):
        q0, k0 = int(st["cu_q"][i]), int(st["cu_k"][i])
        heads = {n: [] for n in names}
        for h in range(hkv):
            q = st["q"][q0:q0 + lq, h * g:(h + 1) * g].double()
            k = st["k"][k0:k0 + lk, h].double()
            v = st["v"][k0:k0 + lk, h].double()
            if case["kind"] == "train":
                seen = torch.arange(lk, device="cuda") <= torch.arange(lk - lq, lk, device="cuda")[:, None]
                got = _exact_rows(q, k, v, st["scale"], seen,
                                  st["d_o"][q0:q0 + lq, h * g:(h + 1) * g].double())
            else:
                # rows in blocks, which bounds the memory
                blocks = []
                for a in range(0, lq, 1024):
                    b = min(lq, a + 1024)
                    if case["kind"] == "attend":
                        seen = (torch.arange(lk, device="cuda")
                                <= torch.arange(lk - lq + a, lk - lq + b, device="cuda")[:, None])
                    else:
                        ids = st["token_ids"][q0 + a:q0 + b].long()
                        seen = torch.zeros(b - a, lk + 1, dtype=torch.bool, device="cuda")
                        seen.scatter_(1, torch.where(ids >= 0, ids, lk), True)
                        seen = seen[:, :lk]
                    blocks.append(_exact_rows(q[a:b], k, v, st["scale"], seen))
                got = [torch.cat(x) for x in zip(*blocks)]
            for n, x in zip(names, got):
                heads[n].append(x)
        for n in names:
            # per-query outputs join along their heads, per-key ones get a head axis
            parts[n].append(torch.stack(heads[n], dim=1) if n in ("dk", "dv")
                            else torch.cat(heads[n], dim=1))
    return {n: torch.cat(parts[n]) for n in names}
