"""Layer norm forward and backward on the GPU against the formulas in 64 bits.

Tolerances are derived from fp32 error bounds, per element.  U = 2^-24 is half
an fp32 step.  A sum of n fp32 terms is off by at most D * U * sum |terms|
with D the longest chain of additions; D = ceil(n / 64) + 16 bounds every way
the kernels may split a row (64 lanes or more, then a tree), D = rows + 16 a
column sum.  Outputs add half a step of their type (finfo.eps / 2).
"""
import pytest
import torch

import fp8_precision_quant_amd as fq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
bf16, f32 = torch.bfloat16, torch.float32
EPS = 1e-5

SHAPES = [(1, 1), (1, 7), (3, 8), (5, 63), (2, 64), (9, 65), (4, 127), (33, 128), (7, 511), (16, 512), (5, 513),
          (130, 1000), (3, 1025), (17, 2047), (4, 2048), (6, 2049), (3, 4095), (300, 4096), (2, 4097), (3, 5003),
          (5, 8192), (3, 8195), (2, 12288), (2, 16384), (3, 16391), (1, 32768), (2, 40001), (1, 65536), (2500, 96)]
TYPES = [(bf16, f32), (bf16, bf16), (f32, f32), (f32, bf16)]


def _rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def _inputs(rows, cols, xt, wt, seed=1, shift=0.5):
    x = _rand(rows, cols, seed=seed) * torch.exp(0.5 * _rand(rows, 1, seed=seed + 1)) + shift
    w = 1 + 0.3 * _rand(cols, seed=seed + 2)
    b = 0.2 * _rand(cols, seed=seed + 3)
    return x.to(xt).to(DEV), w.to(wt).to(DEV), b.to(wt).to(DEV)


def _half(t):
    return torch.finfo(t).eps / 2


def forward_ref(x, w, b, eps=EPS):
    """(y, mean, rstd) in 64 bits and the bounds on the kernel's error of each."""
    xt, cols = x.dtype, x.shape[1]
    x = x.double()
    w = torch.ones(cols, dtype=torch.float64, device=DEV) if w is None else w.double()
    b = torch.zeros(cols, dtype=torch.float64, device=DEV) if b is None else b.double()
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    xh = (x - mean) * rstd
    y = xh * w + b
    D = -(-cols // 64) + 16
    e_mean = (D + 2) * U * x.abs().mean(1, keepdim=True)                  # the sum, then the division
    # the squares: (x - mean) carries e_mean (its own rounding U |x - mean|); around a mean that is off by e the
    # mean square grows by e^2 exactly (the linear term sums to the error of the mean itself)
    rel_var = (D + 6) * U + (2 * e_mean * e_mean + 2 * e_mean * U * x.abs().amax(1, keepdim=True)) / (var + eps)
    rel_rstd = rel_var / 2 + 4 * U
    e_xh = xh.abs() * (rel_rstd + 4 * U) + e_mean * rstd
    e_y = e_xh * w.abs() + 3 * U * (xh * w).abs() + 2 * U * b.abs()
    e_y = 2 * e_y + _half(xt) * (y.abs() + 2 * e_y) + 1e-38
    return (y, mean[:, 0], rstd[:, 0]), (e_y, 2 * e_mean[:, 0] + 1e-38, 2 * (rel_rstd * rstd)[:, 0])


def _check(got, want, tol, what):
    assert got.shape == want.shape, what
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), "%s: %d off, worst %g of the tolerance at %s" % (
        what, int(bad.sum()), float((d / tol).max()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, xt, wt):
    x, w, b = _inputs(rows, cols, xt, wt, seed=rows + cols)
    y, mean, rstd = fq.fp8q_layer_norm_forward(x, w, b, eps=EPS)
    assert y.dtype == xt and mean.dtype == f32 and rstd.dtype == f32
    want, tol = forward_ref(x, w, b)
    for g, r, t, n in zip((y, mean, rstd), want, tol, ("y", "mean", "rstd")):
        _check(g, r, t, n)


@pytest.mark.parametrize("cols", [100, 2048, 9000, 20000])
def test_forward_far_mean(cols):
    """A mean 300 times the deviation: squares around the mean, not a difference of squares."""
    x, w, b = _inputs(4, cols, f32, f32, seed=5, shift=300.0)
    y, mean, rstd = fq.fp8q_layer_norm_forward(x, w, b, eps=EPS)
    want, tol = forward_ref(x, w, b)
    for g, r, t, n in zip((y, mean, rstd), want, tol, ("y", "mean", "rstd")):
        _check(g, r, t, n)


@pytest.mark.parametrize("xt", [bf16, f32])
def test_forward_without_weights_and_constant_rows(xt):
    x = torch.full((3, 333), 2.5, dtype=xt, device=DEV)
    y, mean, rstd = fq.fp8q_layer_norm_forward(x, eps=EPS)
    assert (y == 0).all() and (mean == 2.5).all()
    _check(rstd, torch.full((3,), EPS ** -0.5, dtype=torch.float64, device=DEV), 4 * U * EPS ** -0.5, "rstd")
    x, w, b = _inputs(4, 600, xt, f32, seed=3)
    for ww, bb in ((w, None), (None, b)):
        y, mean, rstd = fq.fp8q_layer_norm_forward(x, ww, bb, eps=EPS)
        want, tol = forward_ref(x, ww, bb)
        _check(y, want[0], tol[0], "y")


def test_non_finite_rows_stay_alone():
    x, w, b = _inputs(5, 700, bf16, f32, seed=9)
    clean = fq.fp8q_layer_norm_forward(x, w, b)[0].clone()
    x[1, 3], x[3, 699] = float("nan"), float("inf")
    y = fq.fp8q_layer_norm_forward(x, w, b)[0]
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all()
    for r in (0, 2, 4):
        assert torch.equal(y[r], clean[r])


def backward_ref(dy, x, mean, rstd, w):
    """(dx, dw, db) in 64 bits and the bounds."""
    xt, (rows, cols) = x.dtype, x.shape
    wt = f32 if w is None else w.dtype
    x, dy, mean, rstd = x.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    w = torch.ones(cols, dtype=torch.float64, device=DEV) if w is None else w.double()
    xh = (x - mean) * rstd                                  # the kernel's: 2 roundings, 3 U
    u = dy * w                                              # one rounding
    c1 = u.mean(1, keepdim=True)
    c2 = (u * xh).mean(1, keepdim=True)
    dx = rstd * (u - c1 - xh * c2)
    D = -(-cols // 64) + 16
    e1 = (D + 4) * U * u.abs().mean(1, keepdim=True)
    e2 = (D + 8) * U * (u * xh).abs().mean(1, keepdim=True)
    e_dx = rstd * (6 * U * (u.abs() + c1.abs()) + e1 + xh.abs() * (e2 + 8 * U * c2.abs()))
    e_dx = 2 * e_dx + _half(xt) * (dx.abs() + 2 * e_dx) + 1e-38
    dw, db = (dy * xh).sum(0), dy.sum(0)
    e_dw = (rows + 16 + 6) * U * (dy * xh).abs().sum(0)
    e_db = (rows + 16) * U * dy.abs().sum(0)
    return (dx, dw, db), (e_dx, e_dw + _half(wt) * (dw.abs() + e_dw) + 1e-38,
                          e_db + _half(wt) * (db.abs() + e_db) + 1e-38)


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES + [(4097, 40), (1025, 1027), (600, 8192), (9000, 1)])
def test_backward(rows, cols, xt, wt):
    x, w, b = _inputs(rows, cols, xt, wt, seed=rows + 3 * cols)
    dy = (0.01 * _rand(rows, cols, seed=77)).to(xt).to(DEV)
    (_, mean, rstd), _ = forward_ref(x, w, b)
    mean, rstd = mean.float(), rstd.float()
    got = fq.fp8q_layer_norm_backward(dy, x, mean, rstd, w)
    assert got[0].dtype == xt and got[1].dtype == wt and got[2].dtype == wt
    want, tol = backward_ref(dy, x, mean, rstd, w)
    for g, r, t, n in zip(got, want, tol, ("dx", "dw", "db")):
        _check(g, r, t, n)


def test_backward_without_weights():
    x, _, _ = _inputs(37, 500, bf16, f32, seed=2)
    dy = _rand(37, 500, seed=78).to(bf16).to(DEV)
    y, mean, rstd = fq.fp8q_layer_norm_forward(x)
    dx, dw, db = fq.fp8q_layer_norm_backward(dy, x, mean, rstd)
    assert dw is None and db is None
    want, tol = backward_ref(dy, x, mean, rstd, None)
    _check(dx, want[0], tol[0], "dx")
    db = torch.empty(500, device=DEV)
    dx, dw, db2 = fq.fp8q_layer_norm_backward(dy, x, mean, rstd, db=db)
    assert dw is None and db2 is db
    _check(db, want[2], tol[2], "db")


def test_empty_batch():
    w = torch.ones(64, device=DEV)
    x = torch.empty(0, 64, dtype=bf16, device=DEV)
    y, mean, rstd = fq.fp8q_layer_norm_forward(x, w, w)
    assert y.shape == (0, 64) and mean.numel() == 0
    dx, dw, db = fq.fp8q_layer_norm_backward(x, x, mean, rstd, w, dw=torch.full((64,), 7.0, device=DEV),
                                             db=torch.full((64,), 7.0, device=DEV))
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("cols", [40, 1000, 4096])
def test_gradients_match_differences(cols):
    """<dx, v>, <dw, v_w> and <db, v_b> against central differences of the kernel's own forward pass."""
    rows, h = 6, 2.0 ** -6
    x, w, b = _inputs(rows, cols, f32, f32, seed=21)
    dy = _rand(rows, cols, seed=22).to(DEV)
    vx, vw, vb = (_rand(rows, cols, seed=23).to(DEV), _rand(cols, seed=24).to(DEV), _rand(cols, seed=25).to(DEV))
    y, mean, rstd = fq.fp8q_layer_norm_forward(x, w, b, eps=EPS)
    got = fq.fp8q_layer_norm_backward(dy, x, mean, rstd, w)
    _, tol = backward_ref(dy, x, mean, rstd, w)
    # the backward takes mean and rstd as fp32: their own error enters the gradient; a bound by evaluating the
    # formula with the 64-bit statistics
    (_, m64, r64), _ = forward_ref(x, w, b)
    exact, _ = backward_ref(dy, x, m64, r64, w)
    stat, _ = backward_ref(dy, x, mean, rstd, w)
    for i, (v, name) in enumerate(((vx, "x"), (vw, "w"), (vb, "b"))):
        args = [x, w, b]
        out, e_out, ref = [], 0.0, []
        for sign in (1, -1):
            moved = list(args)
            moved[i] = args[i] + sign * h * v
            yk = fq.fp8q_layer_norm_forward(*moved, eps=EPS)[0]
            (yr, _, _), (ty, _, _) = forward_ref(*moved)
            out.append((dy.double() * yk.double()).sum())
            ref.append((dy.double() * yr).sum())
            e_out = e_out + (dy.double().abs() * ty).sum()
        step = (torch.add(args[i], v, alpha=h).double() - torch.add(args[i], v, alpha=-h).double()) / (2 * h)
        differences = (out[0] - out[1]) / (2 * h)
        along = (got[i].double() * step).sum()
        truncation = ((ref[0] - ref[1]) / (2 * h) - (exact[i] * step).sum()).abs()
        bound = truncation + e_out / (2 * h) + (step.abs() * (tol[i] + 2 * (stat[i] - exact[i]).abs())).sum()
        assert (along - differences).abs() <= bound, name
        # and the bound says something: it is well below the derivative's size
        assert bound < 0.2 * (got[i].double() * step).abs().sum(), name


@pytest.mark.parametrize("xt", [bf16, f32])
@pytest.mark.parametrize("cols,ld,at", [(100, 131, 1), (2047, 2049, 3), (4096, 4099, 5), (9001, 9010, 1),
                                        (20001, 20003, 1)])
def test_strides_alignment_and_surroundings(cols, ld, at, xt):
    """Rows at any element address and stride give the same bits as packed ones, and nothing around is written."""
    rows = 5
    x, w, b = _inputs(rows, cols, xt, f32, seed=31)
    dy = _rand(rows, cols, seed=32).to(xt).to(DEV)

    def odd(t, fill):
        buf = torch.full((rows * ld + at + 9,), fill, dtype=t.dtype, device=DEV)
        view = buf[at:at + rows * ld].view(rows, ld)[:, :cols]
        if t.numel():
            view.copy_(t)
        return buf, view

    y, mean, rstd = fq.fp8q_layer_norm_forward(x, w, b)
    _, xo = odd(x, float("nan"))
    ybuf, yo = odd(torch.zeros_like(x), -7.0)
    y2, mean2, rstd2 = fq.fp8q_layer_norm_forward(xo, w, b, y=yo)
    assert torch.equal(yo, y) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
    mask = torch.ones_like(ybuf, dtype=torch.bool)
    mask[at:at + rows * ld].view(rows, ld)[:, :cols] = False
    assert (ybuf[mask] == -7.0).all()

    dx, dw, db = fq.fp8q_layer_norm_backward(dy, x, mean, rstd, w)
    _, dyo = odd(dy, float("nan"))
    dbuf, dxo = odd(torch.zeros_like(x), -7.0)
    _, dw2, db2 = fq.fp8q_layer_norm_backward(dyo, xo, mean, rstd, w, dx=dxo)
    assert torch.equal(dxo, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    assert (dbuf[mask] == -7.0).all()


def test_same_bits_every_time_and_other_stream():
    x, w, b = _inputs(777, 1531, bf16, f32, seed=41)
    dy = _rand(777, 1531, seed=42).to(bf16).to(DEV)
    y, mean, rstd = fq.fp8q_layer_norm_forward(x, w, b)
    first = fq.fp8q_layer_norm_backward(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        if stream is not None:
            side.wait_stream(torch.cuda.current_stream())
        again = (*fq.fp8q_layer_norm_forward(x, w, b, stream=stream),
                 *fq.fp8q_layer_norm_backward(dy, x, mean, rstd, w, stream=stream))
        torch.cuda.synchronize()
        for a, g in zip(again, (y, mean, rstd, *first)):
            assert torch.equal(a, g)


def test_more_than_2_31_elements():
    """Offsets past 32 bits: a row stride that puts the last rows beyond 2^32 elements' bytes."""
    rows, cols, ld = 5, 2000, (1 << 29) + 3
    buf = torch.empty(rows * ld, dtype=bf16, device=DEV)
    xo = buf.view(rows, ld)[:, :cols]
    x, w, b = _inputs(rows, cols, bf16, f32, seed=51)
    xo.copy_(x)
    y, mean, rstd = fq.fp8q_layer_norm_forward(x, w, b)
    y2, _, _ = fq.fp8q_layer_norm_forward(xo, w, b)
    assert torch.equal(y, y2)
    dx, dw, db = fq.fp8q_layer_norm_backward(x, x, mean, rstd, w)
    dx2, dw2, db2 = fq.fp8q_layer_norm_backward(x, xo, mean, rstd, w)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)
