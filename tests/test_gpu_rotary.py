"""kpool_rotary, forward and backward, against 64 bits (tolerances: rotary_reference.py)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import check_selection_vs_oracle
from pool_score_top_amd import kpool as K
from pool_score_top_amd import synth
from rotary_reference import check, make, turned

BF16, F32 = torch.bfloat16, torch.float32


def freqs_of(pairs, scale=1.0):
    return K.rotary_frequencies(pairs, scale=scale, trained=4096)


# (rows, heads, D, begin, pairs, pad): whole heads, parts at both ends, every vector width, odd ones
SHAPES = [(1, 1, 2, 0, 1, 0), (7, 3, 64, 0, 32, 0), (33, 1, 128, 0, 32, 0), (130, 4, 192, 128, 32, 0),
          (65, 2, 128, 64, 32, 8), (9, 5, 80, 4, 20, 4), (21, 3, 50, 2, 9, 2), (40, 7, 37, 3, 11, 5),
          (3, 130, 96, 0, 48, 0), (2, 1, 1024, 0, 512, 0), (5, 2, 1023, 1, 511, 1), (300, 1, 16, 8, 4, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,heads,D,begin,pairs,pad", SHAPES)
def test_against_64_bits(rows, heads, D, begin, pairs, pad, dtype, interleaved):
    x, pos = make(rows, heads, D, dtype, rows * D + pairs, pad, 100000)
    freqs, factor = freqs_of(pairs, 8.0)
    how = dict(begin=begin, interleaved=interleaved, factor=factor)
    check(x, K.rotary(x, pos, freqs, **how), pos, freqs, begin, interleaved, factor)
    check(x, K.rotary_backward(x.contiguous(), pos, freqs, **how), pos, freqs, begin, interleaved, factor, -1)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(interleaved):
    x, _ = make(6, 2, 64, F32, 3)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32, device="cuda")
    freqs, factor = freqs_of(32)
    y = K.rotary(x, pos, freqs, interleaved=interleaved)
    check(x, y, pos, freqs, 0, interleaved, factor)
    assert torch.equal(y[0], x[0])


@pytest.mark.gpu
def test_one_head_rows_and_many_rows():
    x, pos = make(70000, 1, 128, BF16, 4, dims=2, far=524288)
    freqs, factor = freqs_of(32, 40.0)
    check(x, K.rotary(x, pos, freqs, factor=factor), pos, freqs, 0, False, factor)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,begin,pairs,pad", [(64, 0, 32, 0), (64, 32, 16, 16), (37, 3, 11, 5)])
def test_in_place_and_slices_equal_a_copy(D, begin, pairs, pad, interleaved):
    x, pos = make(50, 3, D, BF16, 5, pad)
    freqs, _ = freqs_of(pairs)
    how = dict(begin=begin, interleaved=interleaved, factor=1.25)
    ref = K.rotary(x, pos, freqs, **how)
    wide = torch.full((50, 2 * 3 * D + 16), 7.0, dtype=BF16, device="cuda")
    left, right = (wide[:, a:a + 3 * D].unflatten(1, (3, D)) for a in (0, 3 * D + 8))
    left.copy_(x)
    out = K.rotary(left, pos, freqs, out=right, **how)   # side by side in the same rows
    assert out is right and torch.equal(right, ref) and torch.equal(left, x)
    assert (wide[:, 3 * D:3 * D + 8] == 7).all() and (wide[:, 6 * D + 8:] == 7).all()
    K.rotary(left, pos, freqs, out=left, **how)
    assert torch.equal(left, ref) and (wide[:, 3 * D:3 * D + 8] == 7).all()
    bits = lambda t: t.view(torch.int16)
    assert torch.equal(K.rotary(bits(x), pos, freqs, **how), bits(ref))


@pytest.mark.gpu
def test_no_rows():
    freqs, _ = freqs_of(4)
    x = torch.empty(0, 2, 8, dtype=BF16, device="cuda")
    assert K.rotary(x, torch.empty(0, dtype=torch.int32, device="cuda"), freqs).shape == (0, 2, 8)


@pytest.mark.gpu
def test_nan_and_inf_stay_in_their_pair():
    x, pos = make(20, 2, 64, BF16, 6)
    x[3, 1, 5], x[4, 0, 40] = float("nan"), float("inf")
    freqs, _ = freqs_of(16)
    ref = K.rotary(x, pos, freqs)
    clean = x.clone()
    clean[3, 1, 5] = clean[4, 0, 40] = 0.0
    got = K.rotary(clean, pos, freqs)
    touched = torch.zeros_like(x, dtype=torch.bool)
    touched[3, 1, 5] = touched[3, 1, 21] = touched[4, 0, 40] = True
    assert ref[3, 1, 5].isnan() and ref[3, 1, 21].isnan() and ref[4, 0, 40] == float("inf")
    assert torch.equal(ref[~touched], got[~touched])


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_is_the_transpose_and_agrees_with_differences(interleaved):
    """<R x, dy> = <x, R^T dy>; R is linear, so central differences of any step are exact but for
    fp32's roundings of the two sides (D terms of 8 u each)."""
    x, pos = make(11, 2, 48, F32, 7)
    dy, _ = make(11, 2, 48, F32, 8)
    freqs, _ = freqs_of(20)
    how = dict(begin=6, interleaved=interleaved, factor=1.5)
    y, dx = K.rotary(x, pos, freqs, **how).double(), K.rotary_backward(dy, pos, freqs, **how).double()
    slack = 2 * 16 * U32 * 1.5 * (x.double().abs().sum((1, 2)) * dy.double().abs().amax((1, 2)))
    assert ((y * dy.double()).sum((1, 2)) - (x.double() * dx).sum((1, 2))).abs().le(slack).all()
    step = torch.zeros_like(x)
    for at in ((0, 0, 6), (3, 1, 7), (10, 1, 45), (5, 0, 0)):
        step.zero_()[at] = 1.0
        up, down = (K.rotary(x + s * step, pos, freqs, **how).double() for s in (1, -1))
        diff = ((up - down) / 2 * dy.double()).sum()
        # four values of up and down are not their common part: each within 16 u of the largest
        assert abs(float(diff - dx[at])) <= 16 * 16 * U32 * float(x.abs().max() + 1) * float(dy.abs().max())


U32 = 2.0 ** -24


@pytest.mark.gpu
def test_other_stream_and_captured_calls():
    x, pos = make(200, 4, 64, BF16, 9)
    freqs, _ = freqs_of(32)
    ref = K.rotary(x, pos, freqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = K.rotary(x, pos, freqs, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = K.rotary(x, pos, freqs)
        dx = K.rotary_backward(y, pos, freqs)
    for i in range(4):
        x.copy_(make(200, 4, 64, BF16, 50 + i)[0])
        y.fill_(3), dx.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        ref = K.rotary(x, pos, freqs)
        assert torch.equal(y, ref) and torch.equal(dx, K.rotary_backward(ref, pos, freqs))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows 2^26 elements apart, 9 GB of them."""
    rows, wide = 70, 1 << 26
    far = torch.empty(rows * wide, dtype=BF16, device="cuda").view(rows, wide)
    x, pos = make(rows, 2, 64, BF16, 10)
    freqs, _ = freqs_of(32)
    there = far[:, :128].unflatten(1, (2, 64))
    there.copy_(x)
    out = far[:, 256:384].unflatten(1, (2, 64))
    ref = K.rotary(x, pos, freqs)
    assert torch.equal(K.rotary(there, pos, freqs, out=out), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved,norm,gated,q_lo,q_hi", [
    (False, False, False, 0, None), (True, True, False, 0, None), (False, True, True, 0, None),
    (False, True, False, 200, 1100)])
def test_selector_with_rotary_positions(interleaved, norm, gated, q_lo, q_hi):
    """The selection of turned queries and keys by its oracle, on what rotary itself gives."""
    cu = np.array([0, 700, 701, 701, 1500], dtype=np.int32)
    wl = synth.workload("sq4096", T=1500, kpool=4, budget=64)
    r = synth.host_inputs(wl, 3)
    dev = {n: torch.from_numpy(r[n].view(np.int16) if r[n].dtype == np.uint16 else r[n]).cuda() for n in ("q", "k", "w")}
    g = torch.Generator().manual_seed(1)
    k_norm = ((1 + 0.2 * torch.randn(128, generator=g)).cuda(), torch.randn(128, generator=g).cuda(), 1e-6) if norm else None
    freqs, factor = freqs_of(32, 40.0)
    how = dict(begin=64, interleaved=interleaved, factor=factor)
    sel = K.Selector(cu, 4, 64, 32, 128, rotary=(freqs, 64, interleaved, factor), q_lo=q_lo, q_hi=q_hi)
    extra = {}
    if gated:
        extra = dict(g=torch.randn(1500, 128, generator=g).to(BF16).cuda().view(torch.int16),
                     ape=torch.randn(4, 128, generator=g).cuda())
    out = sel.run(dev["q"], dev["k"], dev["w"], k_norm=k_norm, **extra)
    pos = torch.cat([torch.arange(int(b - a)) for a, b in zip(cu[:-1], cu[1:])]).to(torch.int32).cuda()
    keys = K.layer_norm(dev["k"], *k_norm)[0] if norm else dev["k"]
    q, k = K.rotary(dev["q"], pos, freqs, **how), K.rotary(keys, pos, freqs, **how)
    check(dev["q"].view(BF16), q.view(BF16), pos, freqs, 64, interleaved, factor)
    plain = K.Selector(cu, 4, 64, 32, 128, q_lo=q_lo, q_hi=q_hi).run(q, k, dev["w"], **extra)
    assert torch.equal(out["token_ids"], plain["token_ids"]) and torch.equal(out["kp"], plain["kp"])
    if gated or q_hi:
        return
    ref = oracle.select(q.cpu().numpy().view(np.uint16), k.cpu().numpy().view(np.uint16), r["w"], cu, 4, 64)
    cu_pools, _ = oracle.count_pools(cu, 4)
    seq, t = oracle.row_positions(np.arange(1500), cu)
    nvis = oracle.visible_pools(t, 4, cu_pools[seq + 1] - cu_pools[seq])
    check_selection_vs_oracle(out["pool_ids"].cpu().numpy(), ref["scores"], nvis, 64, "rotary")


def test_frequencies():
    freqs, factor = K.rotary_frequencies(32, device="cpu")
    assert factor == 1.0 and freqs.dtype == torch.float64
    assert np.allclose(freqs.numpy(), [10000.0 ** (-j / 32) for j in range(32)], rtol=1e-14)
    linear, factor = K.rotary_frequencies(32, scale=4.0, device="cpu")
    assert factor == 1.0 and torch.equal(linear, freqs / 4)
    mixed, factor = K.rotary_frequencies(32, scale=40.0, trained=4096, device="cpu")
    turns = 4096 * freqs / (2 * np.pi)
    assert factor == pytest.approx(0.1 * np.log(40) + 1)
    assert torch.equal(mixed[turns >= 32], freqs[turns >= 32])
    assert torch.allclose(mixed[turns <= 1], freqs[turns <= 1] / 40, rtol=1e-15)
    between = (turns > 1) & (turns < 32)
    assert between.any() and (mixed[between] < freqs[between]).all() and (mixed[between] > freqs[between] / 40).all()
    for bad in (dict(pairs=0), dict(pairs=4, scale=0.5), dict(pairs=4, base=0.0), dict(pairs=4, scale=2.0, trained=0)):
        with pytest.raises(ValueError):
            K.rotary_frequencies(**bad, device="cpu")


AT = dict(x=1 << 20, pos=1 << 24, freqs=2 << 24, y=3 << 24)


def _call(rows=5, heads=2, D=64, begin=0, pairs=16, factor=1.0, dtype=0, flags=0, xs=None, ys=None, **at):
    at = {**AT, **at}
    p = lambda n: None if at[n] is None else ctypes.c_void_p(at[n])
    return K.lib().kpool_rotary(p("x"), heads * D if xs is None else xs, p("pos"), p("freqs"), rows, heads, D, begin,
                                pairs, factor, dtype, flags, p("y"), heads * D if ys is None else ys, None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(heads=0), dict(heads=65537), dict(D=0), dict(D=1), dict(D=1026), dict(begin=-1), dict(begin=33),
    dict(begin=65), dict(pairs=0), dict(pairs=33), dict(factor=float("nan")), dict(factor=float("inf")), dict(dtype=2),
    dict(flags=4), dict(xs=127), dict(ys=127), dict(xs=1 << 41), dict(x=None), dict(y=None), dict(pos=None),
    dict(freqs=None), dict(x=(1 << 20) + 1), dict(y=(3 << 24) + 1), dict(dtype=1, x=(1 << 20) + 2), dict(pos=(1 << 24) + 2),
    dict(freqs=(2 << 24) + 4)])
def test_refuses(kw):
    assert _call(**kw) == K.KPOOL_EINVAL


@pytest.mark.parametrize("kw", [
    dict(y=AT["x"] + 2), dict(y=AT["x"], xs=128, ys=130), dict(y=AT["x"] + 256, xs=256, ys=255),
    dict(y=AT["x"] + 200, xs=256, ys=256), dict(y=AT["x"] + 300, xs=256, ys=256), dict(y=AT["pos"] - 1000),
    dict(y=AT["freqs"]), dict(y=AT["pos"] + 16 - 4 * 512, ys=256), dict(y=AT["x"] - 512 * 4 + 100, xs=256, ys=256)])
def test_refuses_overlaps(kw):
    assert _call(**kw) == K.KPOOL_EINVAL and b"overlaps" in K.lib().kpool_last_error()


def test_takes_and_refuses_sizes():
    assert _call(rows=0, x=None, y=None, pos=None, freqs=None) == K.KPOOL_OK
    assert _call(rows=(1 << 31) + 1) == K.KPOOL_EUNSUPPORTED
    assert _call(rows=1 << 30, heads=128, xs=1 << 20, ys=1 << 20, y=AT["x"] + 2) == K.KPOOL_EUNSUPPORTED


def test_refuses_in_python():
    x, pos, f = torch.zeros(2, 3, 8), torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.float64)
    with pytest.raises(ValueError, match="device"):
        K.rotary(x, pos, f)
    with pytest.raises(ValueError, match="autograd"):
        K.rotary(x.requires_grad_(), pos, f)


@pytest.mark.gpu
def test_refuses_tensors_of_other_shapes():
    x, pos = make(5, 2, 16, BF16, 1)
    f, _ = freqs_of(4)
    for bad in (lambda: K.rotary(x, pos[:4], f), lambda: K.rotary(x, pos.long(), f), lambda: K.rotary(x, pos, f.float()),
                lambda: K.rotary(x.half(), pos, f), lambda: K.rotary(x.transpose(1, 2), pos, f),
                lambda: K.rotary(x, pos, f, out=x[:4]), lambda: K.rotary(x, pos, f, out=x.float()),
                lambda: K.rotary(x[0, 0], pos, f), lambda: K.rotary(x, pos, f.cpu())):
        with pytest.raises(ValueError):
            bad()


def test_selector_of_a_range_holds_the_queries_of_its_rows():
    cu = np.array([0, 700, 701, 701, 1500], dtype=np.int32)
    freqs, factor = K.rotary_frequencies(32, device="cpu")
    for q_lo, q_hi, rows in ((200, 210, 10), (1490, None, 10), (0, None, 1500), (700, 700, 0)):
        sel = K.Selector(cu, 4, 64, 32, 128, device="cpu", q_lo=q_lo, q_hi=q_hi, rotary=(freqs, 0, False, factor))
        assert sel.q_turned.shape == (rows, 32, 128) and sel.k_turned.shape == (1500, 128)


@pytest.mark.gpu
@pytest.mark.parametrize("q_lo,q_hi", [(0, 3), (699, 705), (1490, 1500), (1499, 1500), (700, 700)])
def test_selector_of_few_rows_equals_the_whole(q_lo, q_hi):
    """Ids of a range of rows against those of all rows; the range's buffers hold no others."""
    cu = np.array([0, 700, 701, 701, 1500], dtype=np.int32)
    wl = synth.workload("sq4096", T=1500, kpool=4, budget=64)
    r = synth.host_inputs(wl, 5)
    q, k, w = (torch.from_numpy(r[n].view(np.int16) if r[n].dtype == np.uint16 else r[n]).cuda() for n in ("q", "k", "w"))
    freqs, factor = freqs_of(32, 40.0)
    make_sel = lambda **kw: K.Selector(cu, 4, 64, 32, 128, rotary=(freqs, 64, True, factor), **kw)
    whole = make_sel().run(q, k, w)
    few = make_sel(q_lo=q_lo, q_hi=q_hi)
    for _ in range(2):
        out = few.run(q, k, w)
        assert torch.equal(out["pool_ids"], whole["pool_ids"][q_lo:q_hi])
        assert torch.equal(out["token_ids"], whole["token_ids"][q_lo:q_hi])


@pytest.mark.gpu
def test_queries_and_weights_outside_the_range_are_not_read():
    cu = np.array([0, 700, 701, 701, 1500], dtype=np.int32)
    r = synth.host_inputs(synth.workload("sq4096", T=1500, kpool=4, budget=64), 6)
    q, k, w = (torch.from_numpy(r[n].view(np.int16) if r[n].dtype == np.uint16 else r[n]).cuda() for n in ("q", "k", "w"))
    whole = K.Selector(cu, 4, 64, 32, 128).run(q, k, w)["token_ids"]
    for lo, hi in ((0, 3), (690, 705), (1499, 1500)):
        outside = torch.ones(1500, dtype=torch.bool, device="cuda")
        outside[lo:hi] = False
        q2, w2 = q.clone(), w.clone()
        q2.view(BF16)[outside], w2[outside] = float("nan"), float("nan")
        out = K.Selector(cu, 4, 64, 32, 128, q_lo=lo, q_hi=hi).run(q2, k, w2)
        assert torch.equal(out["token_ids"], whole[lo:hi])
