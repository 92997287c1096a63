"""Layer norm, forward and backward, against the formulas in 64 bits.

Tolerances (u = 2^-24 is fp32's half step, h the half step of the output's type): a sum of
n terms in fp32, in any order that adds at most `depth` values one after the other, is off
by at most depth * u * sum|terms|.  A thread adds its columns in turn and the lanes join in
a tree, so depth <= N / 16 + 16 covers every layout of the kernels for rows, and the row
sums of the weight's gradient add rows of one workgroup, then the workgroups' sums.
  mean     depth u max|x|                                                  (and u |mean|)
  xh       the mean's error times rstd, and rstd's relative (depth + 8) u
  y        xh's error times |w|, 3 roundings, and h |y| for the output's type
  dx       depth u on each of the two means, a few roundings, and h |dx|
A constant of 2 on the fp32 part covers the products of these errors.
"""
import numpy as np
import pytest
import torch

from pool_score_top_amd import kpool as K

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def forward64(x, w, b, eps):
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = 1.0 / ((xc * xc).mean(1, keepdim=True) + eps).sqrt()
    return xc * rstd * w + b, mean, rstd


def inputs(rows, N, dtype, seed, pad=0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    wide = (torch.randn(rows, N + pad, generator=g) + offset).to(dtype).cuda()
    x = wide[:, :N]
    w = (1.0 + 0.3 * torch.randn(N, generator=g)).cuda()
    b = torch.randn(N, generator=g).cuda()
    dy = torch.randn(rows, N, generator=g).to(dtype).cuda()
    return x, w, b, dy


def check_forward(x, w, b, eps, y, mean, rstd):
    rows, N = x.shape
    x64 = x.double()
    w64 = torch.ones(N, dtype=torch.float64, device="cuda") if w is None else w.double()
    b64 = torch.zeros(N, dtype=torch.float64, device="cuda") if b is None else b.double()
    y64, m64, r64 = forward64(x64, w64, b64, eps)
    depth = N / 16 + 16
    top = x64.abs().amax(1, keepdim=True)
    xh = (x64 - m64) * r64
    tol32 = 2 * U * ((depth + 16) * (w64.abs() * (top * r64 + xh.abs())) + 3 * b64.abs())
    tol = HALF[x.dtype] * (y64.abs() + tol32) + tol32
    assert ((y.double() - y64).abs() <= tol).all()
    if mean is not None:
        assert ((mean.double() - m64[:, 0]).abs() <= 2 * (depth + 2) * U * top[:, 0]).all()
        # the shift of the mean enters the variance squared, relative to it (top rstd depth u)^2
        rel = 2 * ((depth + 8) * U + (depth * U * top * r64) ** 2)[:, 0]
        assert ((rstd.double() - r64[:, 0]).abs() <= rel * r64[:, 0]).all()


def check_backward(x, w, dy, mean, rstd, dx, dw, db):
    """Against the formulas with the kernel's own mean and rstd as inputs."""
    rows, N = x.shape
    x64, g0 = x.double(), dy.double()
    w64 = torch.ones(N, dtype=torch.float64, device="cuda") if w is None else w.double()
    mu, rs = mean.double()[:, None], rstd.double()[:, None]
    xh = (x64 - mu) * rs
    g = g0 * w64
    c1, c2 = (g * xh).mean(1, keepdim=True), g.mean(1, keepdim=True)
    d64 = rs * (g - c2 - xh * c1)
    depth = N / 16 + 16
    a1, a2 = (g * xh).abs().mean(1, keepdim=True), g.abs().mean(1, keepdim=True)
    tol32 = 2 * U * rs * (6 * g.abs() + (depth + 8) * (a2 + xh.abs() * a1))
    tol = HALF[x.dtype] * (d64.abs() + tol32) + tol32
    assert ((dx.double() - d64).abs() <= tol).all()
    depth = 16 * 1024 if rows > 16 * 1024 else rows  # (far above the longest run of any split)
    assert ((dw.double() - (g0 * xh).sum(0)).abs() <= 2 * (depth + 8) * U * (g0 * xh).abs().sum(0)).all()
    assert ((db.double() - g0.sum(0)).abs() <= 2 * (depth + 8) * U * g0.abs().sum(0)).all()


# one vector or less a row, each thread layout and its edges, rows past the registers
WIDTHS = [1, 2, 7, 8, 16, 63, 64, 127, 128, 136, 256, 500, 512, 1000, 1024, 1237, 2048, 2056, 4096,
          4100, 8192, 8200, 9001, 20480]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", WIDTHS)
def test_layer_norm_and_gradients(N, dtype):
    for rows in (1, 5, 67):
        x, w, b, dy = inputs(rows, N, dtype, 100 * N + rows)
        y, mean, rstd = K.layer_norm(x, w, b, 1e-5, want_stats=True)
        check_forward(x, w, b, 1e-5, y, mean, rstd)
        check_backward(x, w, dy, mean, rstd, *K.layer_norm_backward(dy, x, w, mean, rstd))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,pad", [(1, 1), (3, 2), (5, 0), (7, 1), (8, 1), (9, 0), (64, 3), (127, 0), (129, 5), (257, 0),
                                   (513, 1), (1023, 0), (1030, 0), (2049, 0), (4099, 2), (6150, 1), (8192, 1),
                                   (8193, 0), (12289, 0), (16391, 3)])
def test_rows_that_start_and_end_anywhere(N, pad, dtype):
    """Rows at every alignment, whose last vector shares elements with the one before."""
    for rows in (1, 37):
        x, w, b, dy = inputs(rows, N, dtype, 10 * N + rows, pad, offset=1.0)
        y, mean, rstd = K.layer_norm(x, w, b, 1e-5, want_stats=True)
        check_forward(x, w, b, 1e-5, y, mean, rstd)
        grads = K.layer_norm_backward(dy, x, w, mean, rstd)
        check_backward(x, w, dy, mean, rstd, *grads)
        assert all(torch.equal(p, q) for p, q in zip(grads, K.layer_norm_backward(dy, x, w, mean, rstd)))
        again = K.layer_norm(x, w, b, 1e-5)[0]
        assert torch.equal(again, y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,N,pad", [(70001, 128, 0), (70001, 128, 8), (3000, 100, 3), (5000, 640, 16)])
def test_many_rows_and_row_strides(rows, N, pad, dtype):
    """Slices of a wider projection, on the vector path (pad 8, 16) and off it (pad 3)."""
    x, w, b, dy = inputs(rows, N, dtype, 7, pad, offset=2.0)
    y, mean, rstd = K.layer_norm(x, w, b, 1e-6, want_stats=True)
    check_forward(x, w, b, 1e-6, y, mean, rstd)
    check_backward(x, w, dy, mean, rstd, *K.layer_norm_backward(dy, x, w, mean, rstd))


@pytest.mark.gpu
def test_without_weight_and_bias_and_wanted_outputs():
    x, w, b, dy = inputs(37, 129, torch.float32, 3)
    for weight, bias in ((None, None), (w, None), (None, b)):
        y, mean, rstd = K.layer_norm(x, weight, bias, 0.0, want_stats=True)
        check_forward(x, weight, bias, 0.0, y, mean, rstd)
        dx, dw, db = K.layer_norm_backward(dy, x, weight, mean, rstd)
        check_backward(x, weight, dy, mean, rstd, dx, dw, db)
        only = K.layer_norm_backward(dy, x, weight, mean, rstd, want_dweight=False, want_dbias=False)
        assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
        only = K.layer_norm_backward(dy, x, weight, mean, rstd, want_dx=False, want_dweight=False)
        assert only[0] is None and only[1] is None and torch.equal(only[2], db)


@pytest.mark.gpu
def test_constant_and_large_rows():
    """A constant row has variance 0: y is the bias; the formula's NaN only with eps 0.  A row
    with NaN or an infinity spoils no other row."""
    x = torch.full((3, 128), 5.0, device="cuda")
    w, b = torch.full((128,), 2.0, device="cuda"), torch.arange(128.0, device="cuda")
    y, mean, rstd = K.layer_norm(x, w, b, 1e-6, want_stats=True)
    assert torch.equal(y, b.expand(3, 128)) and (mean == 5.0).all()
    assert K.layer_norm(x, w, b, 0.0)[0].isnan().all()
    x, w, b, _ = inputs(64, 128, torch.bfloat16, 5)
    ref = K.layer_norm(x, w, b)[0]
    x = x.clone()
    x[3, 7], x[20, 0] = float("nan"), float("inf")
    y = K.layer_norm(x, w, b)[0]
    keep = torch.ones(64, dtype=torch.bool, device="cuda")
    keep[3] = keep[20] = False
    assert torch.equal(y[keep], ref[keep]) and y[3].isnan().all() and y[20].isnan().all()


@pytest.mark.gpu
def test_gradients_match_differences():
    """dx, dw and db along a random direction against central differences of the 64-bit
    forward: with a step of 1e-5 the cubic term is about 1e-10 and the kernel's fp32 gradients
    are good to 1e-5 of the sums' magnitude."""
    x, w, b, dy = inputs(6, 200, torch.float32, 11)
    _, mean, rstd = K.layer_norm(x, w, b, 1e-5, want_stats=True)
    grads = K.layer_norm_backward(dy, x, w, mean, rstd)
    g = torch.Generator().manual_seed(1)
    p = [x.double(), w.double(), b.double()]
    for i in range(3):
        d = torch.randn(p[i].shape, generator=g, dtype=torch.float64).cuda()
        up, dn = list(p), list(p)
        up[i], dn[i] = p[i] + 1e-5 * d, p[i] - 1e-5 * d
        num = (dy.double() * (forward64(*up, 1e-5)[0] - forward64(*dn, 1e-5)[0])).sum() / 2e-5
        terms = (grads[i].double() * d)
        assert abs(num - terms.sum()) <= 1e-5 * terms.abs().sum()


@pytest.mark.gpu
def test_same_bits_every_time_and_rows_outside_untouched():
    x, w, b, dy = inputs(40000, 128, torch.bfloat16, 9)
    y, mean, rstd = K.layer_norm(x, w, b, want_stats=True)
    a = K.layer_norm_backward(dy, x, w, mean, rstd)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(a, K.layer_norm_backward(dy, x, w, mean, rstd)))
    big = torch.full((40010, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    K.layer_norm(x, w, b, out=big[:40000])
    assert torch.equal(big[:40000], y) and (big[40000:] == 9.0).all()


@pytest.mark.gpu
def test_no_rows():
    x, w, b, dy = inputs(0, 128, torch.bfloat16, 9)
    y, mean, rstd = K.layer_norm(x, w, b, want_stats=True)
    assert y.shape == (0, 128)
    dx, dw, db = K.layer_norm_backward(dy, x, w, mean, rstd)
    assert dx.shape == (0, 128) and (dw == 0).all() and (db == 0).all()


@pytest.mark.gpu
def test_captured_step_replays_equal_eager():
    """Forward and backward in one graph, replayed over new inputs between eager calls, on a
    stream of its own."""
    x, w, b, dy = inputs(999, 640, torch.bfloat16, 21)
    x = x.clone()
    ws = torch.empty(K.layer_norm_backward_workspace_bytes(999, 640), dtype=torch.uint8, device="cuda")

    def step():
        y, mean, rstd = K.layer_norm(x, w, b, want_stats=True)
        return (y, mean, rstd) + K.layer_norm_backward(dy, x, w, mean, rstd, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(inputs(999, 640, torch.bfloat16, 30 + i)[0])
        for t in out:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(p, q) for p, q in zip(got, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = K.layer_norm(x, w, b, stream=side)[0]
    side.synchronize()
    assert torch.equal(y, got[0])


# ---------------------------------------------------------------------------
# Refusals (no GPU: the checks come before any launch)
# ---------------------------------------------------------------------------

def _c(**kw):
    a = dict(x=16, stride=128, w=16, b=16, rows=4, N=128, eps=1e-6, dtype=0, y=32, mean=16, rstd=16)
    a.update(kw)
    return K.lib().kpool_layer_norm(a["x"], a["stride"], a["w"], a["b"], a["rows"], a["N"], a["eps"],
                                    a["dtype"], a["y"], a["mean"], a["rstd"], None)


def _c_bwd(**kw):
    a = dict(dy=16, x=16, stride=128, w=16, mean=16, rstd=16, rows=4, N=128, dtype=0, ws=16,
             ws_bytes=1 << 20, dx=16, dw=16, db=16)
    a.update(kw)
    return K.lib().kpool_layer_norm_backward(a["dy"], a["x"], a["stride"], a["w"], a["mean"], a["rstd"],
                                             a["rows"], a["N"], a["dtype"], a["ws"], a["ws_bytes"],
                                             a["dx"], a["dw"], a["db"], None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(N=0), dict(stride=127), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(dtype=2), dict(x=None), dict(y=None), dict(x=17), dict(y=18, dtype=1),
    dict(w=18), dict(mean=17), dict(y=16), dict(N=(1 << 26) + 1, stride=1 << 30)])
def test_layer_norm_refuses(kw):
    assert _c(**kw) == K.KPOOL_EINVAL
    assert K.lib().kpool_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), K.KPOOL_EINVAL), (dict(N=0), K.KPOOL_EINVAL), (dict(stride=127), K.KPOOL_EINVAL),
    (dict(dtype=-1), K.KPOOL_EINVAL), (dict(dy=None), K.KPOOL_EINVAL), (dict(mean=None), K.KPOOL_EINVAL),
    (dict(dx=None, dw=None, db=None), K.KPOOL_EINVAL), (dict(dy=17), K.KPOOL_EINVAL),
    (dict(ws=24), K.KPOOL_EINVAL), (dict(ws=None), K.KPOOL_EWORKSPACE),
    (dict(ws_bytes=1023), K.KPOOL_EWORKSPACE), (dict(ws_bytes=0, dw=None), K.KPOOL_EWORKSPACE)])
def test_layer_norm_backward_refuses(kw, code):
    assert _c_bwd(**kw) == code
    assert K.lib().kpool_last_error()


def test_no_rows_need_no_pointers():
    assert _c(rows=0, x=None, y=None) == K.KPOOL_OK
    assert _c_bwd(rows=0, dy=None, x=None, mean=None, rstd=None, dw=None, db=None, ws=None) == K.KPOOL_OK


def test_backward_workspace_bytes():
    assert K.layer_norm_backward_workspace_bytes(4, 128) == 2 * 128 * 4
    assert K.layer_norm_backward_workspace_bytes(0, 128) == 2 * 128 * 4
    assert K.layer_norm_backward_workspace_bytes(1 << 30, 128) == 1024 * 2 * 128 * 4
    assert K.layer_norm_backward_workspace_bytes(-1, 128) == 0
    assert K.layer_norm_backward_workspace_bytes(4, 0) == 0


@pytest.mark.parametrize("bad", [
    lambda x: x.half(), lambda x: x[0], lambda x: x.t(), lambda x: x.cpu()])
def test_binding_refuses_other_tensors(bad):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    if torch.cuda.is_available():
        x = x.cuda()
    with pytest.raises(ValueError):
        K.layer_norm(bad(x))


@pytest.mark.gpu
def test_more_rows_than_a_launch():
    """2^23 + 9 rows of 3: two launches."""
    rows = (1 << 23) + 9
    x = torch.randn(rows, 3, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    y, mean, rstd = K.layer_norm(x, eps=1e-3, want_stats=True)
    for part in (slice(0, 1000), slice((1 << 23) - 500, rows)):
        check_forward(x[part], None, None, 1e-3, y[part], mean[part], rstd[part])


@pytest.mark.parametrize("kw", [dict(y=1 << 20), dict(y=(1 << 20) + 3 * 400 + 254), dict(y=(1 << 20) - 1022)])
def test_layer_norm_refuses_y_over_x(kw):
    assert _c(**{**dict(x=1 << 20, stride=200, y=2 << 20), **kw}) == K.KPOOL_EINVAL
    assert b"overlaps" in K.lib().kpool_last_error()


@pytest.mark.parametrize("dx", [1 << 20, 2 << 20, (1 << 20) + 1022, (2 << 20) + 3 * 400 + 254])
def test_layer_norm_backward_refuses_dx_over_inputs(dx):
    assert _c_bwd(dy=1 << 20, x=2 << 20, stride=200, ws=3 << 20, dx=dx, dw=4 << 20, db=5 << 20) == K.KPOOL_EINVAL
    assert b"overlaps" in K.lib().kpool_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,pad", [(3, 0), (41, 0), (61, 3), (82, 0), (336, 0), (1237, 1), (1240, 0), (4100, 0), (9001, 0),
                                   (16404, 0), (20001, 0)])
def test_constant_rows_of_every_width(N, pad, dtype):
    """The mean of N equal numbers is that number, whatever N and 1 / N: y is the bias, rstd
    1 / sqrt(eps), and with eps 0 the formula's NaN and infinity."""
    values = torch.tensor([1000.0, 10001.0, 0.1, -77.7, 3e30, 1.0], device="cuda").to(dtype)
    x = values[:, None].expand(-1, N + pad).contiguous()[:, :N]
    _, w, b, _ = inputs(1, N, dtype, N)
    y, mean, rstd = K.layer_norm(x, w, b, 1e-6, want_stats=True)
    assert torch.equal(mean, values.float())
    assert torch.equal(y, b.to(dtype).expand_as(y))
    # (the root and the division: half a step each, eps itself is given in fp32)
    want = 1.0 / torch.tensor(1e-6, dtype=torch.float32).double().sqrt().item()
    assert ((rstd.double() - want).abs() <= 3 * U * want).all()
    y, _, rstd = K.layer_norm(x, w, b, 0.0, want_stats=True)
    assert y.isnan().all() and (rstd == float("inf")).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,pad", [(100, 0), (123, 1), (1237, 0), (4096, 0), (9000, 3), (20480, 0)])
def test_small_spread_around_a_large_mean(N, pad, dtype):
    """Rows whose mean is thousands of times their spread.  x - mean takes three roundings of its
    own size (x minus the mean's fp32 part, less the rest, and that rest's 2^-24 of 2^-24 of the
    mean), the mean in 64 bits none that counts; rstd is a sum of N squares of those.  The mean
    that is returned is rounded once."""
    x, w, b, _ = inputs(37, N, torch.float32, N)
    x = 10000.0 + x * torch.logspace(-2, 1.5, 37, device="cuda")[:, None]
    wide = torch.zeros(37, N + pad, dtype=dtype, device="cuda")
    wide[:, :N] = x.to(dtype)
    x = wide[:, :N]
    eps = 1e-6
    y, mean, rstd = K.layer_norm(x, w, b, eps, want_stats=True)
    y64, m64, r64 = forward64(x.double(), w.double(), b.double(), eps)
    assert ((mean.double() - m64[:, 0]).abs() <= 1.001 * U * m64[:, 0].abs()).all()
    depth = N / 16 + 16
    assert ((rstd.double() - r64[:, 0]).abs() <= (depth + 8) * U * r64[:, 0]).all()
    xc = (x.double() - m64).abs()
    tol32 = w.double().abs() * r64 * ((depth + 16) * U * xc + 4 * U * U * m64.abs()) + 3 * U * b.double().abs()
    tol = tol32 + HALF[dtype] * (y64.abs() + tol32)
    assert ((y.double() - y64).abs() <= tol).all()


# (addresses 1 MiB apart; the refusals come before any launch)
APART = dict(x=1 << 20, w=2 << 20, b=3 << 20, y=4 << 20, mean=5 << 20, rstd=6 << 20)
BWD_APART = dict(dy=1 << 20, x=2 << 20, w=3 << 20, mean=4 << 20, rstd=5 << 20, ws=6 << 20, dx=7 << 20, dw=8 << 20,
                 db=9 << 20)


@pytest.mark.parametrize("kw", [
    *[{out: APART[n] + 4} for out in ("mean", "rstd") for n in ("x", "w", "b", "y")],
    *[dict(y=APART[n]) for n in ("w", "b")], dict(mean=APART["rstd"]), dict(rstd=APART["mean"] + 12),
    dict(mean=APART["x"] + 3 * 512 + 252, stride=256), dict(y=APART["w"] - 1022), dict(b=APART["y"] + 1020)])
def test_layer_norm_refuses_outputs_over_inputs_and_one_another(kw):
    assert _c(**{**APART, **kw}) == K.KPOOL_EINVAL
    assert b"overlaps" in K.lib().kpool_last_error()


@pytest.mark.parametrize("kw", [
    *[{out: BWD_APART[n]} for out in ("dw", "db", "ws") for n in ("dy", "x", "w", "mean", "rstd", "dx")],
    *[dict(dx=BWD_APART[n]) for n in ("w", "mean", "rstd")], dict(dw=BWD_APART["db"]),
    dict(db=BWD_APART["dw"] + 508), dict(dw=BWD_APART["ws"] + 1020), dict(ws=BWD_APART["db"] - 1008),
    dict(rows=0, dw=BWD_APART["w"])])
def test_layer_norm_backward_refuses_outputs_over_inputs_and_one_another(kw):
    assert _c_bwd(**{**BWD_APART, **kw}) == K.KPOOL_EINVAL
    assert b"overlaps" in K.lib().kpool_last_error()


@pytest.mark.gpu
def test_statistics_in_the_gaps_of_strided_rows():
    """What lies between the rows of a strided input is not the input's."""
    x, w, b, dy = inputs(1, 128, torch.float32, 3)
    wide = torch.zeros(1, 160, device="cuda")
    wide[:, :128] = x
    y, mean, rstd = K.layer_norm(x, w, b, want_stats=True)
    rc = K.lib().kpool_layer_norm(wide.data_ptr(), 160, w.data_ptr(), b.data_ptr(), 1, 128, 1e-6, K.KPOOL_DTYPE_F32,
                                  y.data_ptr(), wide.data_ptr() + 4 * 128, wide.data_ptr() + 4 * 159,
                                  torch.cuda.current_stream().cuda_stream)
    assert rc == K.KPOOL_OK
    assert torch.equal(wide[0, 128], mean[0]) and torch.equal(wide[0, 159], rstd[0]) and torch.equal(wide[:, :128], x)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,code", [(torch.bfloat16, 0), (torch.float32, 1)])
def test_one_row_has_no_pitch(dtype, code):
    """Any row pitch of a single row gives the bits of the contiguous one."""
    x, w, b, dy = inputs(1, 1240, dtype, 4)
    y, mean, rstd = K.layer_norm(x, w, b, 1e-6, want_stats=True)
    dx, _, _ = K.layer_norm_backward(dy, x, w, mean, rstd)
    s = torch.cuda.current_stream().cuda_stream
    y2, dx2, p = torch.empty_like(y), torch.empty_like(dx), lambda t: t.data_ptr()
    for pitch in (1241, 1243, 5000):
        assert K.lib().kpool_layer_norm(p(x), pitch, p(w), p(b), 1, 1240, 1e-6, code, p(y2), None, None, s) == 0
        assert K.lib().kpool_layer_norm_backward(p(dy), p(x), pitch, p(w), p(mean), p(rstd), 1, 1240, code, None, 0,
                                                 p(dx2), None, None, s) == 0
        assert torch.equal(y, y2) and torch.equal(dx, dx2)
