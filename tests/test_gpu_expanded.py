"""kpool_attend_expanded and its backward pass against 64 bits (tolerances: expanded_reference.py)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from attend_reference import cu_of
from expanded_reference import BF16, check, check_backward, make
from pool_score_top_amd import kpool as K


def run(q_lens, k_lens, Hq, Hkv, D, P, seed, backward=True, **kw):
    cu_q, cqd = cu_of(q_lens)
    cu_k, ckd = cu_of(k_lens)
    x = make(cu_q, cu_k, Hq, Hkv, D, P, seed, **kw)
    cu = (cu_q, cqd, cu_k, ckd)
    o, lse = K.attend_expanded(*x, *cu, want_lse=True)
    scale = (D + P) ** -0.5
    check(*x, cu_q, cu_k, scale, o, lse)
    d_o = torch.randn(o.shape, generator=torch.Generator().manual_seed(seed + 1)).to(BF16).cuda()
    if backward:
        check_backward(*x, d_o, o, lse, cu_q, cu_k, scale, *K.attend_expanded_backward(d_o, *x, o, lse, *cu))
    return x, cu, o, lse, d_o


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,P", [(1, 1, 8, 8), (4, 4, 128, 64), (4, 1, 64, 32), (8, 2, 72, 40), (6, 2, 128, 8),
                                        (5, 5, 120, 64), (16, 16, 64, 64), (40, 1, 64, 16)])
def test_packed_prompts(Hq, Hkv, D, P):
    """Lengths around the tiles' edges, an empty sequence, a single token."""
    lens = [1, 31, 0, 32, 33, 63, 64, 65, 257, 300, 2]
    run(lens, lens, Hq, Hkv, D, P, Hq * 1000 + D + P)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,P", [(2, 2, 128, 64), (12, 4, 64, 32), (16, 16, 128, 64)])
def test_chunks_of_prompts(Hq, Hkv, D, P):
    run([5, 100, 0, 1, 260], [50, 1000, 77, 4096, 261], Hq, Hkv, D, P, Hq + D)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 300])
def test_rows_without_keys(rows):
    """More queries than keys: the first rows see nothing; a sequence without any key, one without rows."""
    run([rows, rows, 4, 0], [2, 0, 9, 5], 4, 2, 64, 32, rows)


@pytest.mark.gpu
@pytest.mark.parametrize("D,P", [(128, 64), (64, 32)])
def test_long_prompts_and_shares(D, P):
    """Parts of the walked axes: few heads over long sequences, and many tiles of unequal lengths."""
    run([3000], [3000], 2, 2, D, P, 5)
    run([1500, 70, 700], [1500, 2500, 700], 4, 4, D, P, 6)


@pytest.mark.gpu
def test_many_sequences():
    lens = [int(x) for x in np.random.default_rng(1).integers(0, 12, 200)]
    run(lens, lens, 4, 4, 64, 32, 7)


@pytest.mark.gpu
@pytest.mark.parametrize("D,P", [(64, 32), (128, 64)])
def test_short_units_beside_long_ones(D, P):
    """Shares of keys' units that are cut, and units of a step or two between them."""
    lens = [1300, 5, 130, 1, 64, 300, 1, 129, 40, 257]
    run(lens, lens, 16, 16, D, P, 17)


@pytest.mark.gpu
def test_strided_tokens():
    run([200, 31], [200, 90], 8, 8, 128, 64, 8, pad=24)


@pytest.mark.gpu
def test_scores_of_every_size():
    for gain in (60.0, 1e-3):
        run([300], [300], 2, 1, 128, 64, 9, gain=gain)


@pytest.mark.gpu
def test_contiguous_heads_equal_halves_of_a_projection():
    (q, k, k_pe, v), cu, o, lse, d_o = run([130, 40], [130, 40], 4, 4, 128, 64, 10)
    grads = K.attend_expanded_backward(d_o, q, k, k_pe, v, o, lse, *cu)
    k, v, k_pe = k.contiguous(), v.contiguous(), k_pe.contiguous()
    o2, lse2 = K.attend_expanded(q, k, k_pe, v, *cu, want_lse=True)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    for a, b in zip(grads, K.attend_expanded_backward(d_o, q, k, k_pe, v, o, lse, *cu)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_gradients_agree_with_differences():
    """Along a direction in each input, central differences of <o, d_o> with o in 64 bits."""
    from expanded_reference import full_keys
    (q, k, k_pe, v), (cu_q, cqd, cu_k, ckd), o, lse, d_o = run([40], [40], 4, 2, 64, 32, 11)
    grads = K.attend_expanded_backward(d_o, q, k, k_pe, v, o, lse, cu_q, cqd, cu_k, ckd)
    x = [t[:40].double() for t in (q, k, k_pe, v)]
    unseen = torch.ones(40, 40, dtype=torch.bool, device="cuda").triu(1)

    def loss(q, k, pe, v):
        total = 0.0
        for h in range(4):
            s = 96 ** -0.5 * q[:, h] @ full_keys(k, pe, 0, 40, h // 2).t()
            w = torch.softmax(s.masked_fill(unseen, -math.inf), 1)
            total = total + (w @ v[:, h // 2] * d_o[:, h].double()).sum()
        return total

    g = torch.Generator().manual_seed(12)
    for i in range(4):
        step = torch.randn(x[i].shape, generator=g, dtype=torch.float64).cuda() * 1e-4
        up, down = (loss(*[t + sign * step if n == i else t for n, t in enumerate(x)]) for sign in (1, -1))
        slope = (grads[i].double() * step).sum()
        # the gradient's values are off by four roundings of bf16 at most, in the norm over the direction
        tol = 4 * 2.0 ** -8 * (grads[i].double().norm() * step.norm())
        assert abs(float((up - down) / 2 - slope)) <= float(tol)


@pytest.mark.gpu
def test_same_bits_other_stream_workspace_and_outputs():
    x, cu, o, lse, d_o = run([1500, 40], [1500, 900], 2, 2, 128, 64, 13)
    grads = K.attend_expanded_backward(d_o, *x, o, lse, *cu)
    nf = K.attend_expanded_workspace_bytes(cu[0], cu[2], 2, 2, 128, 64)
    nb = K.attend_expanded_backward_workspace_bytes(cu[0], cu[2], 2, 2, 128, 64)
    assert nf > 0 and nb > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        ws = torch.full((max(nf, nb),), 255, dtype=torch.uint8, device="cuda")
        out = [torch.full_like(t, 3.0) for t in grads]
        o2, l2 = torch.full_like(o, 3.0), torch.full_like(lse, 3.0)
        torch.cuda.synchronize()
        K.attend_expanded(*x, *cu, out=o2, lse=l2, workspace=ws, stream=stream)
        K.attend_expanded_backward(d_o, *x, o, lse, *cu, workspace=ws, stream=stream,
                                   **dict(zip(("dq", "dk", "dk_pe", "dv"), out)))
        torch.cuda.synchronize()
        assert torch.equal(o2, o) and torch.equal(l2, lse) and all(torch.equal(a, b) for a, b in zip(out, grads))
    bits = [t.view(torch.int16) for t in x]
    o2, none = K.attend_expanded(*bits, *cu)
    assert none is None and torch.equal(o2, o.view(torch.int16))


@pytest.mark.gpu
def test_calls_of_two_threads_at_once():
    import threading
    jobs = []
    for seed, D, P in ((18, 128, 64), (19, 64, 24)):
        x, cu, o, lse, d_o = run([700, 40], [700, 300], 4, 4, D, P, seed)
        jobs.append(lambda stream=None, x=x, cu=cu, o=o, lse=lse, d=d_o: [
            *K.attend_expanded(*x, *cu, want_lse=True, stream=stream),
            *K.attend_expanded_backward(d, *x, o, lse, *cu, stream=stream)])
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


@pytest.mark.gpu
def test_captured_step_replays_equal_eager():
    x, cu, o, lse, d_o = run([400, 30], [400, 600], 4, 4, 128, 64, 14)

    def step():
        o, lse = K.attend_expanded(*x, *cu, want_lse=True)
        return (o, lse) + K.attend_expanded_backward(d_o, *x, o, lse, *cu)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        for t, new in zip(x, make(cu[0], cu[2], 4, 4, 128, 64, 50 + i)):
            t.copy_(new)
        for t in got:
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(first, step()))


@pytest.mark.gpu
def test_in_an_autograd_function():
    x, cu, o, lse, d_o = run([90, 5], [90, 5], 4, 4, 64, 32, 15)
    grads = K.attend_expanded_backward(d_o, *x, o, lse, *cu)
    leaves = [t[:95].clone().requires_grad_() for t in x]
    with pytest.raises(ValueError, match="autograd"):
        K.attend_expanded(*leaves, *cu)

    class Attend(torch.autograd.Function):
        @staticmethod
        def forward(ctx, *x):
            o, lse = K.attend_expanded(*x, *cu, want_lse=True)
            ctx.save_for_backward(*x, o, lse)
            return o

        @staticmethod
        def backward(ctx, d_o):
            *x, o, lse = ctx.saved_tensors
            return K.attend_expanded_backward(d_o.contiguous(), *x, o, lse, *cu)

    out = Attend.apply(*leaves)
    out.backward(d_o)
    assert torch.equal(out, o) and all(torch.equal(t.grad, g) for t, g in zip(leaves, grads))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Tokens 2^24 elements apart, 10 GB of them."""
    T, wide = 300, 1 << 24
    cu, dev = cu_of([T])
    x = [t[:T] for t in make(cu, cu, 2, 2, 64, 32, 16)]
    d_o = torch.randn(T, 2, 64, device="cuda").to(BF16)
    far = torch.empty(T * wide, dtype=BF16, device="cuda").view(T, wide)
    there, at = [], 0
    for t in x:
        n = t[0].numel()
        at = at + 256 if at < 768 else wide - 256
        f = far[:, at:at + n].unflatten(1, t.shape[1:]) if t.dim() == 3 else far[:, at:at + n]
        f.copy_(t)
        there.append(f)

    def calls(x):
        o, lse = K.attend_expanded(*x, cu, dev, want_lse=True)
        return (o, lse) + K.attend_expanded_backward(d_o, *x, o, lse, cu, dev)

    assert all(torch.equal(a, b) for a, b in zip(calls(x), calls(there)))


@pytest.mark.gpu
def test_the_layer_both_ways():
    """A latent attention layer as it is used: positions on queries and keys, the prompt by the expanded form;
    the same projections absorbed give the same rows over the cache of latent rows, whole and over what
    the indexer selected (every visible token here).

    The absorbed queries and outputs pass one more rounding to bf16 each way, q's relative 2^-8 in every
    score: a weight is off by 2 h sum |s_r| relative, s_r the scores' terms over the rank, and the output
    by that and its own roundings."""
    T, H, D, R, P = 150, 8, 64, 128, 32
    g = torch.Generator().manual_seed(17)
    n = lambda *s: torch.randn(*s, generator=g).cuda()
    c = n(T, R).to(BF16)                                   # latent rows
    up_k, up_v = (n(H, D, R) * R ** -0.5 for _ in range(2))
    q = (n(T, H, D + P)).to(BF16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freqs, factor = K.rotary_frequencies(P // 2)
    K.rotary(q, pos, freqs, begin=D, interleaved=True, out=q)
    k_pe = K.rotary(n(T, P).to(BF16), pos, freqs, interleaved=True)
    k = torch.matmul(c.float(), up_k.flatten(0, 1).t().contiguous()).unflatten(1, (H, D)).to(BF16)
    v = torch.matmul(c.float(), up_v.flatten(0, 1).t().contiguous()).unflatten(1, (H, D)).to(BF16)
    cu, dev = cu_of([T])
    scale = (D + P) ** -0.5
    o, lse = K.attend_expanded(q, k, k_pe, v, cu, dev, scale=scale, want_lse=True)
    check(q, k, k_pe, v, cu, cu, scale, o, lse)
    # absorbed: the keys' projection on the queries, the values' on the outputs
    qa = torch.stack([torch.matmul(q[:, h, :D].float(), up_k[h]) for h in range(H)], 1)
    qa = torch.cat([qa.to(BF16), q[:, :, D:]], 2)
    cache = torch.cat([c, k_pe], 1)
    where = dict(k_starts=torch.zeros(1, dtype=torch.int32, device="cuda"))
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    ol, lse_l = K.attend_latent(qa, cache, R, cu, dev, lens, T, scale, want_lse=True, **where)
    ids = torch.where(pos[None] <= pos[:, None], pos[None].expand(T, T), -1).to(torch.int32).contiguous()
    os_, lse_s = K.attend_latent_selected(qa, cache, R, ids, cu, dev, lens, scale, want_lse=True, **where)
    from latent_reference import check as check_latent
    check_latent(qa, [cache], [T], [T], R, scale, ol, lse_l)
    check_latent(qa, [cache], [T], [T], R, scale, os_, lse_s, ids)
    h8 = 2.0 ** -8
    for h in range(H):
        got = torch.matmul(ol[:, h].double(), up_v[h].double().t().contiguous())
        terms = scale * (qa[:, h, :R].double().abs() @ c.double().abs().t() + q[:, h, :D].double().abs() @ k[:, h].double().abs().t())
        seen = pos[None] <= pos[:, None]
        off = torch.where(seen, terms, 0.0).amax(1, keepdim=True) * h8       # of a score, both ways' roundings
        w = torch.softmax(torch.where(seen, scale * (q[:, h, :D].double() @ k[:, h].double().t()
                                                     + q[:, h, D:].double() @ k_pe.double().t()), -math.inf), 1)
        spread = (w @ c.double().abs()) @ up_v[h].double().abs().t() + w @ v[:, h].double().abs()
        assert ((got - o[:, h].double()).abs() <= (2 * off.expm1().clamp(max=1e3) + 6 * h8) * spread).all()


# ---------------------------------------------------------------------------
# Refusals (no GPU)
# ---------------------------------------------------------------------------

AT = dict(q=1 << 32, k=2 << 32, pe=3 << 32, v=4 << 32, cqd=5 << 32, ckd=6 << 32, ws=7 << 32, o=8 << 32, lse=9 << 32,
          d_o=10 << 32, dq=11 << 32, dk=12 << 32, dpe=13 << 32, dv=14 << 32)


def _call(backward=False, cu_q=(0, 10), cu_k=(0, 100), Hq=4, Hkv=2, D=64, P=32, qs=None, ks=None, kh=None, ps=None, vs=None,
          vh=None, scale=0.1, nb=1 << 50, nseq=None, **at):
    at = {**AT, **at}
    p = lambda n: None if at[n] is None else ctypes.c_void_p(at[n])
    cu_q, cu_k = (np.asarray(c, dtype=np.int32) for c in (cu_q, cu_k))
    vp = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    keys = (p("q"), Hq * (D + P) if qs is None else qs, p("k"), Hkv * D if ks is None else ks, D if kh is None else kh,
            p("pe"), P if ps is None else ps, p("v"), Hkv * D if vs is None else vs, D if vh is None else vh)
    cu = (vp(cu_q), p("cqd"), vp(cu_k), p("ckd"), len(cu_q) - 1 if nseq is None else nseq, Hq, Hkv, D, P, scale, p("ws"), nb)
    if backward:
        return K.lib().kpool_attend_expanded_backward(p("d_o"), *keys, p("o"), p("lse"), *cu, p("dq"), p("dk"), p("dpe"),
                                                      p("dv"), None)
    return K.lib().kpool_attend_expanded(*keys, *cu, p("o"), p("lse"), None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(Hq=0), -1), (dict(Hq=5), -1), (dict(D=12), -1), (dict(D=136), -2), (dict(P=0), -1), (dict(P=12), -1),
    (dict(P=72), -2), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(qs=4 * 96 - 8), -1), (dict(qs=388), -1),
    (dict(ks=120), -1), (dict(kh=56), -1), (dict(kh=68), -1), (dict(kh=(1 << 24) + 8), -1), (dict(vh=72), -1),
    (dict(vs=120), -1), (dict(ps=24), -1), (dict(ps=36), -1), (dict(ps=(1 << 24) + 8), -1), (dict(q=None), -1),
    (dict(k=None), -1), (dict(pe=None), -1), (dict(v=None), -1), (dict(o=None), -1), (dict(cqd=None), -1),
    (dict(q=(1 << 32) + 8), -1), (dict(pe=(3 << 32) + 8), -1), (dict(lse=(9 << 32) + 2), -1), (dict(cqd=(5 << 32) + 2), -1),
    (dict(cu_q=(0, 5, 4), cu_k=(0, 5, 6)), -1), (dict(nseq=0), -1)])
def test_refuses(backward, kw, code):
    assert _call(backward, **kw) == code


def test_refuses_workspaces_and_gradients():
    assert _call(cu_k=(0, 50000), nb=16) == -3 and _call(True, nb=16) == -3 and _call(True, ws=None) == -3
    for name in ("d_o", "lse", "dq", "dk", "dpe", "dv"):
        assert _call(True, **{name: None}) == -1
    for name in ("d_o", "dq", "dk", "dpe", "dv", "ws"):
        assert _call(True, **{name: AT[name] + 8}) == -1
    assert _call(True, cu_q=(0, 0), cu_k=(0, 0), q=None, o=None) == 0 and _call(cu_q=(0, 0)) == 0


@pytest.mark.parametrize("backward,out", [(False, "o"), (False, "lse"), (False, "ws"), (True, "dq"), (True, "dk"), (True, "dpe"),
                                          (True, "dv"), (True, "ws")])
@pytest.mark.parametrize("over", ["q", "k", "pe", "v", "cqd", "ckd", "d_o", "o", "lse", "dq", "dk", "dpe", "dv"])
def test_refuses_overlaps(backward, out, over):
    if out == over or (not backward and over in ("d_o", "dq", "dk", "dpe", "dv")):
        return
    assert _call(backward, cu_k=(0, 50000), cu_q=(0, 10), **{out: AT[over]}) == -1
    assert b"overlaps" in K.lib().kpool_last_error()


def test_workspace_bytes_refuse():
    for f in (K.attend_expanded_workspace_bytes, K.attend_expanded_backward_workspace_bytes):
        for bad in ((4, 3, 64, 32), (4, 4, 60, 32), (4, 4, 64, 0), (4, 4, 64, 72)):
            with pytest.raises(K.KpoolError):
                f([0, 5], [0, 5], *bad)


@pytest.mark.gpu
def test_refuses_in_python():
    cu, dev = cu_of([10])
    q, k, k_pe, v = make(cu, cu, 4, 2, 64, 32, 18)
    K.attend_expanded(q, k, k_pe, v, cu, dev)
    for bad in ((q[..., :64], k, k_pe, v), (q, k[..., :56], k_pe, v), (q, k, k_pe[:, :24], v), (q, k, k_pe, v[:, :1]),
                (q, k, k_pe[:9], v), (q.float(), k, k_pe, v), (q, k, k_pe.float(), v), (q, k, k_pe[:, None], v),
                (q, k.transpose(1, 2), k_pe, v)):
        with pytest.raises(ValueError):
            K.attend_expanded(*bad, cu, dev)
