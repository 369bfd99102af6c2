"""The operators' two ways in (plain calls, marshalled natively; calls with a
stream or outputs given, in Python) give the same bits, types and strides, and
every operator can be captured: a graph of a training step's calls is replayed
several times, with eager work of the same tensors and synchronizations in
between, and each replay is compared with the eager result."""
import pytest
import torch

import fp8_precision_quant_amd as fq
from gpu_util import DEV

pytestmark = pytest.mark.gpu

bf16, f32 = torch.bfloat16, torch.float32


def _randn(*shape, seed, dtype=f32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DEV, dtype)


def _same(plain, given):
    plain, given = (t if isinstance(t, tuple) else (t,) for t in (plain, given))
    assert len(plain) == len(given)
    for p, g in zip(plain, given):
        assert (p is None) == (g is None)
        if p is not None:
            assert p.dtype == g.dtype and p.shape == g.shape and p.stride() == g.stride() and p.device == g.device
            assert torch.equal(p, g) and not p.requires_grad


@pytest.mark.parametrize("rows,cols", [(1, 4096), (1, 33), (5, 1), (7, 100), (64, 2048), (300, 1001)])
@pytest.mark.parametrize("dtype,wdtype", [(bf16, f32), (f32, f32), (bf16, bf16)])
def test_norm_and_quantizer(rows, cols, dtype, wdtype):
    big = _randn(rows, cols + 13, seed=1, dtype=dtype)
    for x in (_randn(rows, cols, seed=2, dtype=dtype), big[:, 5:5 + cols]):
        w, b = _randn(cols, seed=3, dtype=wdtype), _randn(cols, seed=4, dtype=wdtype)
        dy = _randn(rows, cols, seed=5, dtype=dtype)
        st = dict(stream=torch.cuda.current_stream())
        for ww, bb in ((w, b), (w, None), (None, b), (None, None)):
            _same(fq.fp8q_layer_norm_forward(x, ww, bb), fq.fp8q_layer_norm_forward(x, ww, bb, **st))
        _, mean, rstd = fq.fp8q_layer_norm_forward(x, w, b)
        _same(fq.fp8q_layer_norm_backward(dy, x, mean, rstd, w), fq.fp8q_layer_norm_backward(dy, x, mean, rstd, w, **st))
        _same(fq.fp8q_int8_quant_rows(x), fq.fp8q_int8_quant_rows(x, **st))


@pytest.mark.parametrize("M,N,K", [(1, 100, 64), (40, 130, 1000), (257, 300, 2048)])
@pytest.mark.parametrize("out", [bf16, f32])
def test_product(M, N, K, out):
    (a, sa), (b, sb) = fq.fp8q_int8_quant_rows(_randn(M, K, seed=1)), fq.fp8q_int8_quant_rows(_randn(N, K, seed=2))
    for bias in (None, _randn(N, seed=3)):
        kw = dict(bias=bias, out_dtype=out)
        _same(fq.fp8q_int8_gemm(a, sa, b, sb, **kw), fq.fp8q_int8_gemm(a, sa, b, sb, stream=torch.cuda.current_stream(), **kw))


@pytest.mark.parametrize("kind", [fq.STATE_F32, fq.STATE_E4M3])
@pytest.mark.parametrize("missing", [False, True])
def test_adamw(kind, missing):
    def run(**kw):
        params = [_randn(n, seed=n) for n in (1, 127, 128, 1000, 0, 4097)] + [_randn(9, 33, seed=7)]
        plan = fq.fp8q_adamw_plan(params, kind)
        for step in range(1, 4):
            grads = [_randn(*p.shape, seed=50 * step + i, dtype=bf16) for i, p in enumerate(params)]
            if missing:
                grads[1] = None
            fq.fp8q_adamw_multi_step(plan, grads if step > 1 else tuple(grads), lr=1e-2, weight_decay=0.1, step=step, **kw)
        return (*params, *plan.moments)
    _same(run(), run(stream=torch.cuda.current_stream()))


@pytest.mark.parametrize("given", [False, True])
def test_a_dropped_plan_waits_for_its_step(given):
    """The memory a plan allocated is not handed out again while a step on another stream may still read it."""
    n = 1 << 20
    params, grads = [_randn(n, seed=1)], [_randn(n, seed=2)]
    want = [p.clone() for p in params]
    fq.fp8q_adamw_multi_step(fq.fp8q_adamw_plan(want), grads, lr=1e-2, step=1)
    torch.cuda.synchronize()
    plan = fq.fp8q_adamw_plan(params)
    owned = {t.data_ptr(): t.numel() * t.element_size() for t in plan._owned}
    side = torch.cuda.Stream()
    x = _randn(2048, 2048, seed=3)
    with torch.cuda.stream(side):
        for _ in range(50):         # the side stream's own work, in front of the step
            x = x @ x
            x = x / x.norm()
    if given:
        fq.fp8q_adamw_multi_step(plan, grads, lr=1e-2, step=1, stream=side)
    else:
        with torch.cuda.stream(side):
            fq.fp8q_adamw_multi_step(plan, grads, lr=1e-2, step=1)
    del plan
    again = [torch.full((b,), 255, dtype=torch.uint8, device=DEV) for b in owned.values()]
    reused = not side.query() and any(t.data_ptr() in owned for t in again)
    side.synchronize()
    assert not reused
    _same(tuple(params), tuple(want))


def test_plain_calls_run_on_the_current_stream():
    x, w = _randn(2000, 4096, seed=1, dtype=bf16), _randn(4096, seed=2)
    want = fq.fp8q_layer_norm_forward(x, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = x.float() * 1.0
        got = fq.fp8q_layer_norm_forward(big.to(bf16), w)
        q = fq.fp8q_int8_quant_rows(got[0])
    side.synchronize()
    _same(want, got)
    _same(fq.fp8q_int8_quant_rows(want[0]), q)


def test_refusals_of_plain_calls():
    x = _randn(4, 64, seed=1)
    with pytest.raises(fq.Fp8qError, match="UNSUPPORTED"):
        fq.fp8q_layer_norm_forward(x, eps=-1.0)
    with pytest.raises(ValueError):
        fq.fp8q_layer_norm_forward(x, _randn(63, seed=2))
    with pytest.raises(ValueError):
        fq.fp8q_layer_norm_forward(x, _randn(64, seed=2).cpu())
    with pytest.raises(ValueError):
        fq.fp8q_layer_norm_forward(x.to(torch.float16))
    with pytest.raises(fq.Fp8qError, match="SHAPE"):
        fq.fp8q_layer_norm_forward(x[:, :0])
    q, s = fq.fp8q_int8_quant_rows(x)
    with pytest.raises(ValueError):
        fq.fp8q_int8_gemm(q, s, q[:, :32], s)
    with pytest.raises(ValueError):
        fq.fp8q_int8_gemm(q, s, q, s.double())
    with pytest.raises(fq.Fp8qError, match="ALIGN"):
        fq.fp8q_int8_gemm(q[:, 1:33], s, q[:, 1:33], s)
    p = [_randn(10, seed=1)]
    plan = fq.fp8q_adamw_plan(p)
    with pytest.raises(fq.Fp8qError, match="UNSUPPORTED"):
        fq.fp8q_adamw_multi_step(plan, [_randn(10, seed=2)], lr=1e-3, step=0)
    with pytest.raises(ValueError):
        fq.fp8q_adamw_multi_step(plan, [_randn(11, seed=2)], lr=1e-3, step=1)


def test_graph_of_a_training_step():
    rows, cols, inner = 300, 1000, 520
    x, dy = _randn(rows, cols, seed=1, dtype=bf16), _randn(rows, cols, seed=2, dtype=bf16)
    w0, b0 = _randn(cols, seed=3), _randn(cols, seed=4)
    w, b = w0.clone(), b0.clone()
    wq, ws = fq.fp8q_int8_quant_rows(_randn(inner, cols, seed=5))
    plan = fq.fp8q_adamw_plan([w, b], fq.STATE_E4M3)

    def step():
        y, mean, rstd = fq.fp8q_layer_norm_forward(x, w, b)
        z = fq.fp8q_int8_gemm(*fq.fp8q_int8_quant_rows(y), wq, ws)
        dx, dw, db = fq.fp8q_layer_norm_backward(dy, x, mean, rstd, w)
        fq.fp8q_adamw_multi_step(plan, [dw, db], lr=1e-2, weight_decay=0.1, step=5)
        return y, z, dx, dw, db

    def reset():
        w.copy_(w0)
        b.copy_(b0)
        for m in plan.moments:
            m.zero_()

    reset()
    want = [t.clone() for t in step()] + [t.clone() for t in (w, b, *plan.moments)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
    for i in range(4):
        reset()
        for t in out:
            t.zero_()
        fq.fp8q_layer_norm_forward(dy, w, b)         # eager work of the same tensors between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (g, r) in enumerate(zip((*out, w, b, *plan.moments), want)):
            assert torch.equal(g, r), "replay %d, output %d" % (i, k)
