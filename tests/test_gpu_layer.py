"""The layer as it is used: index keys normalised, pooled, scored, selected, expanded, and the
attention over what was selected, through Selector.run(k_norm=) and Selector.attend.

Each step is checked against its own reference on the step's actual inputs: the normalised keys
against the library's own layer_norm (which test_gpu_norm.py checks), the selection by its
oracle on those keys, the attention against 64 bits over the token ids that the selection gave
(tolerances: attend_reference.py)."""
import numpy as np
import pytest
import torch

import oracle
from attend_reference import check, make, sequences
from gpu_helpers import check_selection_vs_oracle
from pool_score_top_amd import kpool as K
from pool_score_top_amd import synth

BF16 = torch.bfloat16


def layer(cu, kpool, budget, seed, Hq=8, Hkv=2, D=64, tail=False, q_lo=0, q_hi=None):
    wl = synth.workload("sq4096", T=int(cu[-1]), kpool=kpool, budget=budget)
    r = synth.host_inputs(wl, seed)
    dev = {n: torch.from_numpy(r[n].view(np.int16) if r[n].dtype == np.uint16 else r[n]).cuda()
           for n in ("q", "k", "w")}
    g = torch.Generator().manual_seed(seed)
    norm = ((1 + 0.2 * torch.randn(128, generator=g)).cuda(), torch.randn(128, generator=g).cuda(), 1e-6)
    sel = K.Selector(cu, kpool, budget, 32, 128, tail=tail, q_lo=q_lo, q_hi=q_hi)
    out = sel.run(dev["q"], dev["k"], dev["w"], k_norm=norm)
    cu = np.asarray(cu)
    qkv = [t[:int(cu[-1])] for t in make(cu, cu, Hq, Hkv, D, seed + 1)]
    o, lse = sel.attend(*qkv, want_lse=True)
    return sel, r, dev, norm, out, qkv, o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("cu,kpool,budget,tail", [
    ([0, 700, 701, 701, 1500], 4, 64, False), ([0, 700, 701, 701, 1500], 4, 64, True),
    ([0, 1003], 1, 200, False), ([0, 300, 1200], 5, 7, False), ([0, 90, 400], 4, 128, False),
    ([0, 90, 401], 4, 128, True)])
def test_the_layer(cu, kpool, budget, tail):
    sel, r, dev, norm, out, (q, k, v), o, lse = layer(cu, kpool, budget, 3, tail=tail)
    k_n = K.layer_norm(dev["k"], *norm)[0]
    bits = k_n.cpu().numpy().view(np.uint16)
    ref = oracle.select(r["q"], bits, r["w"], np.asarray(cu, np.int32), kpool, budget, tail=tail)
    np.testing.assert_array_equal(out["kp"].cpu().numpy().view(np.uint16), ref["kp"])
    cu_pools, _ = oracle.count_pools(cu, kpool, tail=tail)
    seq, t = oracle.row_positions(np.arange(cu[-1]), cu)
    nvis = oracle.visible_pools(t, kpool, cu_pools[seq + 1] - cu_pools[seq])
    check_selection_vs_oracle(out["pool_ids"].cpu().numpy(), ref["scores"], nvis, budget, "layer")
    check(q, k, v, np.asarray(cu), np.asarray(cu), 1.0 / 8, o, lse, out["token_ids"])


@pytest.mark.gpu
def test_whole_attention_where_everything_is_selected():
    """budget pools cover every sequence: the lists name every visible token, and both ways of
    the attention agree with 64 bits over them."""
    cu = [0, 90, 400]
    sel, _, _, _, out, (q, k, v), o, lse = layer(cu, 4, 128, 5)
    assert sel.max_pools <= sel.budget
    for a, b, _, _ in sequences(cu, cu):
        ids = out["token_ids"][a:b].long().sort(1).values
        want = torch.arange(b - a, device="cuda")
        assert torch.equal((ids[:, :, None] == want).any(1), want <= want[:, None])
    (cu_q, cu_k), (cqd, ckd) = sel.attend_cu, sel.attend_cu_dev
    by_list = K.attend_selected(q, k, v, out["token_ids"], cu_q, cqd, cu_k, ckd, want_lse=True)
    for got in ((o, lse), by_list):
        check(q, k, v, np.asarray(cu), np.asarray(cu), 1.0 / 8, *got, out["token_ids"])


@pytest.mark.gpu
@pytest.mark.parametrize("budget", [32, 400])
def test_row_ranges_equal_the_whole(budget):
    """Ranges that cut sequences: their rows' tokens are the whole batch's, bit for bit, and the
    attention of them (whose sums run in another order) obeys the same bounds."""
    cu = [0, 300, 1000, 1500]
    sel, _, _, _, out, qkv, o, lse = layer(cu, 4, budget, 7)
    for lo, hi in ((0, 200), (200, 1100), (1100, 1500), (650, 651), (1500, 1500)):
        part = layer(cu, 4, budget, 7, q_lo=lo, q_hi=hi)
        assert torch.equal(part[4]["token_ids"], out["token_ids"][lo:hi])
        assert part[6].shape == (hi - lo, 8, 64)
        cu_q, cu_k = part[0].attend_cu
        check(qkv[0][lo:hi], qkv[1], qkv[2], cu_q, cu_k, 1.0 / 8, part[6], part[7], part[4]["token_ids"])


@pytest.mark.gpu
def test_captured_layer_replays_equal_eager():
    cu = [0, 500, 900]
    sel, _, dev, norm, out, (q, k, v), o, lse = layer(cu, 4, 32, 9)

    def step():
        out = sel.run(dev["q"], dev["k"], dev["w"], k_norm=norm)
        return (out["token_ids"],) + sel.attend(q, k, v, want_lse=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        dev["k"].copy_(torch.from_numpy(synth.host_inputs(synth.workload("sq4096", T=900), 40 + i)["k"]
                                        .view(np.int16)))
        for t in got:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(first, step()))


@pytest.mark.gpu
def test_normed_keys_have_one_place():
    """Rows behind the batch are left out, types of the same bits share the buffer, and other
    keys are refused."""
    cu = [0, 100, 333]
    sel, _, dev, norm, out, _, _, _ = layer(cu, 4, 32, 11)
    ids, place = out["token_ids"].clone(), sel.k_normed.data_ptr()
    k = dev["k"]
    wide = torch.cat([k, torch.full((5, 128), float("nan"), device="cuda").to(BF16).view(k.dtype)])
    for keys in (wide, k.view(BF16), torch.cat([wide, wide], 1)[:, :128]):
        got = sel.run(dev["q"], keys, dev["w"], k_norm=norm)
        assert torch.equal(got["token_ids"], ids) and sel.k_normed.data_ptr() == place
    for bad in (k[:332], k.view(BF16).float(), k[:, :64], k[None]):
        with pytest.raises(ValueError):
            sel.run(dev["q"], bad, dev["w"], k_norm=norm)


def test_row_range():
    cu_q, cu_k = K.row_range([0, 300, 1000, 1500], 200, 1100)
    assert cu_q.tolist() == [0, 100, 800, 900] and cu_k.tolist() == [0, 300, 1000, 1100]
    cu_q, cu_k = K.row_range([0, 300, 1000], 300, 300)
    assert cu_q.tolist() == [0, 0, 0] and cu_k.tolist() == [0, 300, 300]
    for lo, hi in ((-1, 3), (4, 3), (0, 1001)):
        with pytest.raises(ValueError):
            K.row_range([0, 300, 1000], lo, hi)


@pytest.mark.gpu
def test_calls_of_two_threads_at_once():
    """Each on its own stream, with other sizes: the same bits as alone."""
    import threading
    from attend_reference import cu_of

    def work(n, Hq, seed):
        cu, dev = cu_of([n, n // 3])
        q, k, v = make(cu, cu, Hq, 2, 64, seed)
        g = torch.Generator().manual_seed(seed)
        T = int(cu[-1])
        ids = torch.randint(-1, n, (T, 150), generator=g, dtype=torch.int32).cuda()
        d_o = torch.randn(T, Hq, 64, generator=g).to(BF16).cuda()
        x = torch.randn(T, 301, generator=g).to(BF16).cuda()

        def call(stream=None):
            kw = dict(stream=stream)
            o, lse = K.attend(q, k, v, cu, dev, want_lse=True, **kw)
            y, mean, rstd = K.layer_norm(x, want_stats=True, **kw)
            return [o, lse, *K.attend_backward(d_o, q, k, v, o, lse, cu, dev, **kw),
                    *K.attend_selected(q, k, v, ids, cu, dev, want_lse=True, **kw),
                    *K.layer_norm_backward(y, x, None, mean, rstd, **kw)]
        return call

    jobs = [work(700, 4, 1), work(1500, 8, 2)]
    alone = [job() for job in jobs]
    torch.cuda.synchronize()
    wrong = []

    def run(job, want):
        stream = torch.cuda.Stream()
        for _ in range(10):
            got = job(stream)
            stream.synchronize()
            wrong.extend(i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b))

    threads = [threading.Thread(target=run, args=pair) for pair in zip(jobs, alone)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.gpu
def test_profiles_of_the_layer_and_of_the_selection_are_apart():
    """A program that knows the selection's five kinds collects into five entries, whatever else ran
    on its thread; the layer's calls have two entries of their own."""
    import ctypes
    cu = [0, 300, 500]
    sel, _, dev, norm, _, (q, k, v), _, _ = layer(cu, 4, 32, 13)
    K.profile_collect()
    K.profile_enable(True)
    try:
        for _ in range(3):
            sel.run(dev["q"], dev["k"], dev["w"], k_norm=norm)
            sel.attend(q, k, v)
    finally:
        K.profile_enable(False)

    def collect(fn):
        ms, n = (ctypes.c_double * 16)(*[7.0] * 16), (ctypes.c_int64 * 16)(*[7] * 16)
        assert getattr(K.lib(), fn)(ms, n) == K.KPOOL_OK
        return list(ms), list(n)

    ms, n = collect("kpool_profile_collect")
    assert n == [10, 10, 10, 10, 7] + [7] * 11 and ms[4:] == [7.0] * 12
    assert all(t > 7.0 for t in ms[:4])
    ms, n = collect("kpool_layer_profile_collect")
    assert n == [10, 10] + [7] * 14 and all(t > 7.0 for t in ms[:2]) and ms[2:] == [7.0] * 14
    assert set(x[1] for x in K.profile_collect().values()) == {0}


@pytest.mark.parametrize("which", range(3))
def test_refuses_to_lose_gradients(which):
    """Autograd records none of the calls: with tensors that require gradients they raise, on any
    device, before anything else."""
    x = [torch.zeros(2, 1, 8), torch.zeros(2, 1, 8), torch.zeros(2, 1, 8)]
    x[which].requires_grad_()
    cu, cud = np.array([0, 2]), torch.zeros(2, dtype=torch.int32)
    rows = [torch.zeros(2, 8), torch.zeros(8), torch.zeros(8)]
    rows[which].requires_grad_()
    for call in (lambda: K.attend(*x, cu, cud), lambda: K.layer_norm(*rows),
                 lambda: K.attend_selected(*x, torch.zeros(2, 1, dtype=torch.int32), cu, cud)):
        with pytest.raises(ValueError, match="autograd"):
            call()


@pytest.mark.gpu
def test_parameters_without_autograd():
    """The same tensors under no_grad, and in the forward of an autograd function whose backward is
    attend_backward; the selection's key norm, whose ids have no gradients, takes parameters anywhere."""
    from attend_reference import cu_of
    cu, dev = cu_of([70, 5])
    q, k, v = (t[:75].clone() for t in make(cu, cu, 4, 2, 64, 19))
    ref, lse = K.attend(q, k, v, cu, dev, want_lse=True)
    d_o = torch.randn(75, 4, 64, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    grads = K.attend_backward(d_o, q, k, v, ref, lse, cu, dev)

    class Attend(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v):
            o, lse = K.attend(q, k, v, cu, dev, want_lse=True)
            ctx.save_for_backward(q, k, v, o, lse)
            return o

        @staticmethod
        def backward(ctx, d_o):
            return K.attend_backward(d_o.contiguous(), *ctx.saved_tensors, cu, dev)

    x = [t.clone().requires_grad_() for t in (q, k, v)]
    with torch.no_grad():
        assert torch.equal(K.attend(*x, cu, dev)[0], ref)
    o = Attend.apply(*x)
    o.backward(d_o)
    assert torch.equal(o, ref) and all(torch.equal(t.grad, g) for t, g in zip(x, grads))
    sel, _, dev_in, norm, out, _, _, _ = layer([0, 100, 333], 4, 32, 11)
    ids = out["token_ids"].clone()
    params = tuple(torch.nn.Parameter(t) for t in norm[:2]) + norm[2:]
    got = sel.run(dev_in["q"], dev_in["k"], dev_in["w"], k_norm=params)
    assert torch.equal(got["token_ids"], ids) and not got["kp"].requires_grad
