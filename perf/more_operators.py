"""Cases and plain forms of the operators of a latent attention layer around the selection.

Four paths, as a program with such a layer runs them:

  rotary    rotary positions of queries or keys: part of each head, both pair layouts, frequencies
            scaled for long contexts; forward, or forward and backward
  expanded  latent attention with its keys and values expanded for each head and the positional
            part of the keys shared by all heads (prompts), or its training step
  latent    the absorbed form: new tokens' queries over a cache of one latent row a token
  selected  the same over the token ids that the selection gave

`own` is False for the plain forms (elementary torch operations in fp32, angles in fp64,
rounded once at the end) and True for the library's kernels.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # index queries and keys of one serving step: a batch of requests, one new token each
        {"name": "rotary_token", "kind": "rotary", "rows": 8, "heads": 32, "d": 128, "begin": 0, "pairs": 32,
         "interleaved": False, "scaled": 40.0, "type": "bf16", "far": 524288, "pad": 0, "backward": False},
        # index queries of a chunk of a long prompt, half of each head rotated
        {"name": "rotary_index", "kind": "rotary", "rows": 32768, "heads": 32, "d": 128, "begin": 0,
         "pairs": 32, "interleaved": False, "scaled": 40.0, "type": "bf16", "far": 524288, "pad": 0, "backward": False},
        # a training step: the positional end of each query head, in pairs of neighbours
        {"name": "rotary_train", "kind": "rotary", "rows": 8192, "heads": 16, "d": 192, "begin": 128,
         "pairs": 32, "interleaved": True, "scaled": 1.0, "type": "bf16", "far": 8192, "pad": 0, "backward": True},
        # a long prompt read in one pass
        {"name": "expanded_prompt", "kind": "expanded", "q_lens": "8192", "k_lens": "8192", "h": 16, "d": 128,
         "p": 64},
        # a training step over packed documents
        {"name": "expanded_train", "kind": "expanded_train", "q_lens": "4096,2001,511,1",
         "k_lens": "4096,2001,511,1", "h": 16, "d": 128, "p": 64},
        # a training step of a small model: narrow heads, short documents
        {"name": "expanded_small", "kind": "expanded_train", "q_lens": "300,77", "k_lens": "300,77", "h": 8,
         "d": 64, "p": 32},
        # one new token of one short request: the smallest call, where latency counts
        {"name": "latent_token", "kind": "latent", "q_lens": "1", "k_lens": "1003", "h": 16, "r": 512, "p": 64,
         "page": 64},
        # one serving step of a batch of requests, ragged caches in pages, few heads a GPU
        {"name": "latent_batch", "kind": "latent", "q_lens": ",".join(["1"] * 16),
         "k_lens": "32768,30011,28000,24001,20000,16385,16000,12345,9000,8192,4096,2049,1023,130,64,1",
         "h": 16, "r": 512, "p": 64, "page": 64},
        # the same with all heads on the GPU and two new tokens a request (a drafted one behind it)
        {"name": "latent_heads", "kind": "latent", "q_lens": "2,2,2,2,2,2,2,2",
         "k_lens": "32768,30011,24001,16385,9000,4096,1023,65", "h": 128, "r": 512, "p": 64, "page": 16},
        # one new token over what it selected: the smallest call
        {"name": "latent_selected_token", "kind": "selected", "q_lens": "1", "k_lens": "4099", "h": 16, "r": 512,
         "p": 64, "page": 64, "kpool": 4, "budget": 128},
        # one serving step over selected tokens, one new token per request
        {"name": "latent_selected_batch", "kind": "selected", "q_lens": "1,1,1,1,1,1,1,1",
         "k_lens": "65536,50001,32768,20000,10007,4096,900,1", "h": 64, "r": 512, "p": 64, "page": 64, "kpool": 4,
         "budget": 512},
        # a chunk of a 64k-token prompt, each row over the 2048 tokens (512 pools of 4) it selected
        {"name": "latent_selected_rows", "kind": "selected", "q_lens": "1024", "k_lens": "65536", "h": 64,
         "r": 512, "p": 64, "page": 0, "kpool": 4, "budget": 512},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rotary", "expanded", "expanded_train", "latent", "latent", "selected", "selected"])
    if kind == "rotary":
        d = rng.choice([64, 80, 128, 192])
        pairs = rng.choice([d // 2, d // 4, 32 if d >= 128 else 16, 9])
        heads = rng.choice([1, 3, 8, 16, 32])
        return {"kind": "rotary", "rows": _log_int(rng, 1, 134_217_728 // 2 // (heads * d)), "heads": heads, "d": d,
                "begin": rng.choice([0, d - 2 * pairs]), "pairs": pairs, "interleaved": rng.random() < 0.5,
                "scaled": rng.choice([1.0, 4.0, 40.0]), "type": rng.choice(["bf16", "bf16", "f32"]),
                "far": _log_int(rng, 100, 1_000_000), "pad": rng.choice([0, 0, 8, 5]),
                "backward": rng.random() < 0.5}
    if kind in ("expanded", "expanded_train"):
        d, p = rng.choice([(128, 64), (128, 64), (64, 32), (96, 40)])
        h = rng.choice([1, 2, 5, 8, 16])
        if kind == "expanded_train" or rng.random() < 0.5:
            q = [_log_int(rng, 1, 3000) for _ in range(rng.randint(1, 4))]
            k = q
        else:
            q = [_log_int(rng, 1, 600) for _ in range(rng.randint(1, 4))]
            k = [n + _log_int(rng, 1, 8000) for n in q]
        return {"kind": kind, "q_lens": ",".join(map(str, q)), "k_lens": ",".join(map(str, k)), "h": h, "d": d,
                "p": p}
    r, p = rng.choice([(512, 64), (512, 64), (512, 64), (256, 32)])
    h = rng.choice([1, 8, 16, 20, 32, 64, 128])
    page = rng.choice([0, 1, 16, 64, 64, 100])
    if kind == "latent":
        n = rng.randint(1, 8)
        q = [rng.choice([1, 1, 1, 2, 4]) for _ in range(n)]
        k = [a + _log_int(rng, 1, 24000) for a in q]
        return {"kind": "latent", "q_lens": ",".join(map(str, q)), "k_lens": ",".join(map(str, k)), "h": h, "r": r,
                "p": p, "page": page}
    n = rng.randint(1, 4)
    q = [_log_int(rng, 1, 100) for _ in range(n)]
    k = [a + _log_int(rng, 1, 20000) for a in q]
    kpool = rng.choice([1, 2, 4, 5])
    return {"kind": "selected", "q_lens": ",".join(map(str, q)), "k_lens": ",".join(map(str, k)), "h": h, "r": r,
            "p": p, "page": page, "kpool": kpool, "budget": _log_int(rng, 1, 2048 // kpool)}


def _lens(text):
    return [int(x) for x in text.split(",")]


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def work(case):
    if case["kind"] == "rotary":
        size = 2 if case["type"] == "bf16" else 4
        rows, passes = case["rows"], 2 if case["backward"] else 1
        return {"bytes": passes * (2 * rows * case["heads"] * case["d"] * size + 4 * rows) + 8 * case["pairs"],
                "flops": passes * 6 * rows * case["heads"] * case["pairs"]}
    q, k = _lens(case["q_lens"]), _lens(case["k_lens"])
    h, tq, tk = case["h"], sum(q), sum(k)
    if case["kind"] in ("expanded", "expanded_train"):
        d, p = case["d"], case["p"]
        pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(q, k))
        rows, keys = tq * h * (2 * d + p) * 2, tk * (2 * h * d + p) * 2
        if case["kind"] == "expanded":
            return {"bytes": rows + keys + 4 * tq * h, "flops": 2 * (2 * d + p) * h * pairs}
        # (and the gradients: d_o with the rows, dq, dk, dk_pe, dv)
        return {"bytes": 2 * rows + 2 * keys + 4 * tq * h,
                "flops": (2 * (2 * d + p) + 2 * (3 * (d + p) + 2 * d)) * h * pairs}
    r, p = case["r"], case["p"]
    rows = tq * h * (2 * r + p) * 2
    if case["kind"] == "latent":
        pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(q, k))
        return {"bytes": rows + tk * (r + p) * 2 + 4 * tq * h, "flops": 2 * (2 * r + p) * h * pairs}
    width = case["kpool"] * case["budget"]
    pairs = sum(min(width, b - a + i + 1) for a, b in zip(q, k) for i in range(a))
    read = sum(min(b, width * a) for a, b in zip(q, k)) * (r + p) * 2
    return {"bytes": rows + read + 4 * tq * width + 4 * tq * h, "flops": 2 * (2 * r + p) * h * pairs}


def _frequencies(pairs, scaled, trained=4096, base=10000.0, fast=32.0, slow=1.0):
    """Radians a token in fp64, and the factor on the rotated values.  Scaled for contexts `scaled` times
    as long: pairs that turn more than `fast` times within the trained length stay, those that
    turn less than `slow` times are slowed by `scaled`, the others lie between."""
    f = base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    if scaled == 1.0:
        return f, 1.0
    keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
    return f * (keep + (1.0 - keep) / scaled), 0.1 * math.log(scaled) + 1.0


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

    kind = case["kind"]
    if kind == "rotary":
        rows, heads, d = case["rows"], case["heads"], case["d"]
        freqs, factor = _frequencies(case["pairs"], case["scaled"])
        dtype = _TYPES[case["type"]]
        wide = normal(rows, heads * d + case["pad"]).to(dtype)
        st = {"case": case, "x": wide[:, :heads * d].unflatten(1, (heads, d)), "freqs": freqs.cuda(), "factor": factor,
              "positions": torch.randint(0, case["far"], (rows,), device="cuda", generator=gen, dtype=torch.int32)}
        if case["backward"]:
            st["dy"] = normal(rows, heads, d).to(dtype)
        return st
    import numpy as np
    bf16 = torch.bfloat16
    q, k = _lens(case["q_lens"]), _lens(case["k_lens"])
    h, tq, tk = case["h"], sum(q), sum(k)
    st = {"case": case, "cu_q": np.array(_cu(q), dtype=np.int32)}
    st["cu_q_dev"] = torch.from_numpy(st["cu_q"]).cuda()
    if kind in ("expanded", "expanded_train"):
        d, p = case["d"], case["p"]
        st["scale"] = 1.0 / math.sqrt(d + p)
        st["cu_k"] = np.array(_cu(k), dtype=np.int32)
        st["cu_k_dev"] = torch.from_numpy(st["cu_k"]).cuda()
        # (queries a little longer than the keys, so that some scores stand out)
        st["q"] = (2.0 * normal(tq, h, d + p)).to(bf16)
        kv = normal(tk, h, 2 * d).to(bf16)   # the up-projection's output, keys and values of a head side by side
        st["k"], st["v"] = kv[:, :, :d], kv[:, :, d:]
        st["k_pe"] = normal(tk, p).to(bf16)
        if kind == "expanded_train":
            st["d_o"] = normal(tq, h, d).to(bf16)
        return st
    r, p, page = case["r"], case["p"], case["page"]
    st["scale"] = 1.0 / math.sqrt(192.0)  # (of the heads before the projections were absorbed)
    st["q"] = normal(tq, h, r + p).to(bf16)
    st["lens"] = torch.tensor(k, dtype=torch.int32, device="cuda")
    st["max_len"] = max(k)
    if page:
        per = [-(-n // page) for n in k]
        total = sum(per) + 3
        st["cache"] = normal(total, page, r + p).to(bf16)
        free = torch.randperm(total, device="cuda", generator=gen).to(torch.int32)
        table = torch.zeros(len(k), max(per), dtype=torch.int32, device="cuda")
        at = 0
        for s, n in enumerate(per):
            table[s, :n] = free[at:at + n]
            at += n
        st["page_table"] = table
    else:
        st["cache"] = normal(tk, r + p).to(bf16)
        st["starts"] = torch.tensor(_cu(k)[:-1], dtype=torch.int32, device="cuda")
    if kind == "selected":
        st["token_ids"] = _pool_ids(gen, q, k, case["kpool"], case["budget"])
    return st


def _turned(x, st, sign):
    """x with its pairs turned by sign * angle, in fp32, rounded once."""
    case = st["case"]
    begin, n = case["begin"], case["pairs"]
    angle = torch.remainder(st["positions"].double()[:, None] * st["freqs"], 2 * math.pi)
    c = (st["factor"] * angle.cos()).float()[:, None]
    s = (sign * st["factor"] * angle.sin()).float()[:, None]
    y = x.float()
    part = y[:, :, begin:begin + 2 * n]
    if case["interleaved"]:
        a, b = part[:, :, 0::2], part[:, :, 1::2]
        turned = torch.stack([a * c - b * s, a * s + b * c], dim=3).flatten(2)
    else:
        a, b = part[:, :, :n], part[:, :, n:]
        turned = torch.cat([a * c - b * s, a * s + b * c], dim=2)
    return torch.cat([y[:, :, :begin], turned, y[:, :, begin + 2 * n:]], dim=2).to(x.dtype)


def _softmax(s):
    """Weights and log sum exp along the last axis; rows of -inf give zeros."""
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    w = (s - m).exp()
    total = w.sum(dim=-1, keepdim=True)
    lse = (m + total.log()).squeeze(-1)
    return w / torch.where(total > 0, total, torch.ones_like(total)), lse


def _expanded(st):
    case, scale = st["case"], st["scale"]
    d = case["d"]
    q_lens, k_lens = _lens(case["q_lens"]), _lens(case["k_lens"])
    train = case["kind"] == "expanded_train"
    parts = {n: [] for n in (["o", "lse", "dq", "dk", "dk_pe", "dv"] if train else ["o", "lse"])}
    for i, (lq, lk) in enumerate(zip(q_lens, k_lens)):
        q0, k0 = int(st["cu_q"][i]), int(st["cu_k"][i])
        q = st["q"][q0:q0 + lq].float().transpose(0, 1).contiguous()                  # [h, lq, d + p]
        pe = st["k_pe"][k0:k0 + lk].float()
        k = torch.cat([st["k"][k0:k0 + lk].float(), pe[:, None].expand(-1, case["h"], -1)], dim=2)
        k = k.transpose(0, 1).contiguous()                                            # [h, lk, d + p]
        v = st["v"][k0:k0 + lk].float().transpose(0, 1).contiguous()
        unseen = torch.arange(lk, device=q.device) > torch.arange(lk - lq, lk, device=q.device)[:, None]
        s = torch.matmul(q, k.transpose(1, 2).contiguous()).mul_(scale).masked_fill_(unseen, -math.inf)
        w, lse = _softmax(s)
        del s
        parts["o"].append(torch.matmul(w, v).transpose(0, 1))
        parts["lse"].append(lse.t())
        if not train:
            continue
        e = st["d_o"][q0:q0 + lq].float().transpose(0, 1).contiguous()
        dw = torch.matmul(e, v.transpose(1, 2).contiguous())
        ds = w * (dw - (w * dw).sum(dim=2, keepdim=True)) * scale
        dk = torch.matmul(ds.transpose(1, 2).contiguous(), q).transpose(0, 1)
        parts["dq"].append(torch.matmul(ds, k).transpose(0, 1))
        parts["dk"].append(dk[:, :, :d])
        parts["dk_pe"].append(dk[:, :, d:].sum(dim=1))
        parts["dv"].append(torch.matmul(w.transpose(1, 2).contiguous(), e).transpose(0, 1))
    return {n: torch.cat(x).to(torch.float32 if n == "lse" else torch.bfloat16) for n, x in parts.items()}


def _rows_of(st, s, tokens):
    """Cache rows, as they are stored, of a sequence's tokens."""
    if "page_table" in st:
        page = st["case"]["page"]
        rows = st["page_table"][s].long()[tokens // page] * page + tokens % page
        return st["cache"].flatten(0, 1)[rows]
    return st["cache"][st["starts"][s].long() + tokens]


def _latent(st):
    case, scale, r = st["case"], st["scale"], st["case"]["r"]
    q_lens, k_lens = _lens(case["q_lens"]), _lens(case["k_lens"])
    o, lse = [], []
    for i, (lq, lk) in enumerate(zip(q_lens, k_lens)):
        q0 = int(st["cu_q"][i])
        q = st["q"][q0:q0 + lq].float()
        if case["kind"] == "latent":
            c = _rows_of(st, i, torch.arange(lk, device=q.device)).float()
            unseen = torch.arange(lk, device=q.device) > torch.arange(lk - lq, lk, device=q.device)[:, None]
            s = torch.matmul(q.flatten(0, 1), c.t().contiguous()).unflatten(0, (lq, case["h"])).mul_(scale)
            w, l = _softmax(s.masked_fill_(unseen[:, None], -math.inf))
            o.append(torch.matmul(w.flatten(0, 1), c[:, :r].contiguous()).unflatten(0, (lq, case["h"])))
            lse.append(l)
            continue
        for a in range(0, lq, 128):  # (in blocks of rows: the gathered rows are what fills the memory)
            ids = st["token_ids"][q0 + a:q0 + min(lq, a + 128)].long()
            c = _rows_of(st, i, ids.clamp(min=0)).float()                           # [rows, width, r + p]
            s = torch.matmul(q[a:a + 128], c.transpose(1, 2).contiguous()).mul_(scale)
            w, l = _softmax(s.masked_fill_((ids < 0)[:, None], -math.inf))
            o.append(torch.matmul(w, c[:, :, :r].contiguous()))
            lse.append(l)
    return {"o": torch.cat(o).to(torch.bfloat16), "lse": torch.cat(lse)}


def run(state):
    st, kind = state, state["case"]["kind"]
    if not own:
        if kind == "rotary":
            out = {"y": _turned(st["x"], st, 1.0)}
            if st["case"]["backward"]:
                out["dx"] = _turned(st["dy"], st, -1.0)
            return out
        return _expanded(st) if kind in ("expanded", "expanded_train") else _latent(st)
    from pool_score_top_amd import kpool as K
    if kind == "rotary":
        how = dict(begin=st["case"]["begin"], interleaved=st["case"]["interleaved"], factor=st["factor"])
        out = {"y": K.rotary(st["x"], st["positions"], st["freqs"], **how)}
        if st["case"]["backward"]:
            out["dx"] = K.rotary_backward(st["dy"], st["positions"], st["freqs"], **how)
        return out
    if kind in ("expanded", "expanded_train"):
        cu = (st["cu_q"], st["cu_q_dev"], st["cu_k"], st["cu_k_dev"])
        keys = (st["q"], st["k"], st["k_pe"], st["v"])
        o, lse = K.attend_expanded(*keys, *cu, scale=st["scale"], want_lse=True)
        if kind == "expanded":
            return {"o": o, "lse": lse}
        dq, dk, dk_pe, dv = K.attend_expanded_backward(st["d_o"], *keys, o, lse, *cu, scale=st["scale"])
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dk_pe": dk_pe, "dv": dv}
    where = dict(page_table=st.get("page_table"), k_starts=st.get("starts"), scale=st["scale"], want_lse=True)
    cu = (st["cu_q"], st["cu_q_dev"])
    if kind == "latent":
        o, lse = K.attend_latent(st["q"], st["cache"], st["case"]["r"], *cu, st["lens"], st["max_len"], **where)
    else:
        o, lse = K.attend_latent_selected(st["q"], st["cache"], st["case"]["r"], st["token_ids"], *cu, st["lens"],
                                          **where)
    return {"o": o, "lse": lse}


def _exact_rotary(x, st, conjugate):
    """The pairs as complex numbers times factor * e^(i angle), in 64 bits."""
    case = st["case"]
    b, n = case["begin"], case["pairs"]
    turn = torch.polar(torch.full((), st["factor"], dtype=torch.float64, device="cuda").expand(case["rows"], n).contiguous(),
                       torch.outer(st["positions"].double(), st["freqs"]))
    if conjugate:
        turn = turn.conj()
    i = torch.arange(n, device="cuda")
    first, second = (b + 2 * i, b + 2 * i + 1) if case["interleaved"] else (b + i, b + n + i)
    out = x.double()
    z = torch.complex(out[..., first], out[..., second]) * turn[:, None]
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_heads(q, k, v, scale, seen, d_o=None):
    """One head in 64 bits: q [rows, w], k [keys, w], v [keys, d], seen [rows, keys]."""
    s = (scale * q @ k.t()).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, dim=1)
    w = torch.exp(s - lse[:, None])
    o = w @ v
    if d_o is None:
        return o, lse
    dsc = scale * w * (d_o @ v.t() - (d_o * o).sum(1, keepdim=True))
    return o, lse, dsc @ k, dsc.t() @ q, w.t() @ d_o


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "rotary":
        out = {"y": _exact_rotary(st["x"], st, False)}
        if case["backward"]:
            out["dx"] = _exact_rotary(st["dy"], st, True)
        return out
    q_lens, k_lens, h = _lens(case["q_lens"]), _lens(case["k_lens"]), case["h"]
    k_at = _cu(k_lens)
    blocks = {}

    def put(name, x):
        blocks.setdefault(name, []).append(x)

    for i, (lq, lk) in enumerate(zip(q_lens, k_lens)):
        q0 = int(st["cu_q"][i])
        t = torch.arange(lk - lq, lk, device="cuda")
        if case["kind"] in ("expanded", "expanded_train"):
            keys = slice(k_at[i], k_at[i] + lk)
            heads = []
            for j in range(h):
                q = st["q"][q0:q0 + lq, j].double()
                k = torch.cat([st["k"][keys, j], st["k_pe"][keys]], dim=1).double()
                v = st["v"][keys, j].double()
                if case["kind"] == "expanded_train":
                    seen = torch.arange(lk, device="cuda") <= t[:, None]
                    heads.append(_exact_heads(q, k, v, st["scale"], seen, st["d_o"][q0:q0 + lq, j].double()))
                    continue
                rows = []
                for a in range(0, lq, 2048):   # rows in blocks, which bounds the memory
                    seen = torch.arange(lk, device="cuda") <= t[a:a + 2048, None]
                    rows.append(_exact_heads(q[a:a + 2048], k, v, st["scale"], seen))
                heads.append([torch.cat(x) for x in zip(*rows)])
            got = [torch.stack(x, dim=1) for x in zip(*heads)]
            put("o", got[0])
            put("lse", got[1])
            if case["kind"] == "expanded_train":
                d = case["d"]
                put("dq", got[2])
                put("dk", got[3][:, :, :d])
                put("dk_pe", got[3][:, :, d:].sum(1))
                put("dv", got[4])
            continue
        # every token's cache row, found one page at a time
        if case["page"]:
            pages = st["page_table"][i, :-(-lk // case["page"])].tolist()
            c = torch.cat([st["cache"][n] for n in pages])[:lk].double()
        else:
            c = st["cache"][k_at[i]:k_at[i] + lk].double()
        for a in range(lq):
            if case["kind"] == "latent":
                mine = c[:int(t[a]) + 1]
            else:
                ids = st["token_ids"][q0 + a]
                mine = c[ids[ids >= 0].long()]
            seen = torch.ones(1, 1, dtype=torch.bool, device="cuda")
            o, lse = _exact_heads(st["q"][q0 + a].double(), mine, mine[:, :case["r"]], st["scale"], seen)
            put("o", o[None])
            put("lse", lse[None])
    return {n: torch.cat(x) for n, x in blocks.items()}
