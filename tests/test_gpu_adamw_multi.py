"""The AdamW step over many tensors on the GPU.

The step is a fixed sequence of fp32 roundings, so it is checked bit for bit
against the CPU oracle per tensor (E4M3 and fp32 moments), against the
one-tensor entry point, and against the formulas in 64 bits with bounds from
the number of roundings.
"""
import numpy as np
import pytest
import torch

import fp8_precision_quant_amd as fq
import oracle
import synthetic
from gpu_util import DEV, host

pytestmark = pytest.mark.gpu

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)
U = 2.0 ** -24
KINDS = [fq.STATE_E4M3, fq.STATE_F32]

# the sizes where a block, a chunk of 4096 or a vector of four ends, one before and after
SIZES = [1, 0, 3, 5, 127, 128, 129, 4095, 4096, 4097, 255, 8192, 12289, 2, 70001]


def _grad(n, seed, dtype):
    g = synthetic.normal_f32((max(n, 1),), seed, 1e-3)[:n]
    t = torch.from_numpy(g.copy())
    return t.to(dtype)


def _case(sizes, kind, gdtype, seed):
    """Parameters, gradients and moments on the host (numpy), and the same on the GPU as the call takes them."""
    ps, gs, ms = [], [], []
    for i, n in enumerate(sizes):
        p, _, m, v = synthetic.adam_inputs(max(n, 1), seed + i)
        p, m, v = p[:n], m[:n], v[:n]
        ps.append(p)
        gs.append(_grad(n, seed + 100 + i, gdtype))
        if kind == fq.STATE_E4M3:
            if n:
                mq, s1 = oracle.quant_1x128(m[None, :])
                vq, s2 = oracle.quant_1x128(v[None, :])
                ms.append((mq[0], s1[0], vq[0], s2[0]))
            else:
                z8, z4 = np.zeros(0, np.uint8), np.zeros(0, np.float32)
                ms.append((z8, z4, z8, z4))
        else:
            ms.append((m, v))
    dp = [torch.from_numpy(p.copy()).to(DEV) for p in ps]
    dg = [g.to(DEV) for g in gs]
    plan = fq.fp8q_adamw_plan(dp, kind)
    for i, n in enumerate(sizes):
        _put(plan, i, ms[i])
    return ps, [g.float().numpy() for g in gs], ms, dp, dg, plan


def _parts(plan, i):
    """Views of tensor i's moments."""
    b, n = plan.blocks[i], plan.sizes[i]
    nb = -(-n // 128)
    if plan.kind == fq.STATE_F32:
        return tuple(t[b * 128:b * 128 + n] for t in plan.moments)
    mq, ms, vq, vs = plan.moments
    return mq[b * 128:b * 128 + n], ms[b:b + nb], vq[b * 128:b * 128 + n], vs[b:b + nb]


def _put(plan, i, values):
    for view, v in zip(_parts(plan, i), values):
        view.copy_(torch.from_numpy(np.ascontiguousarray(v)))


def _oracle_step(p, g, state, kind, wd, t):
    if p.size == 0:
        return p, state
    if kind == fq.STATE_E4M3:
        out = oracle.adamw_fp8_step(p, g, *state, HP["lr"], HP["beta1"], HP["beta2"], HP["eps"], wd, t)
    else:
        out = oracle.adamw_step(p, g, *state, HP["lr"], HP["beta1"], HP["beta2"], HP["eps"], wd, t)
    return out[0], tuple(out[1:])


def _same(a, b, what):
    a, b = np.ascontiguousarray(a), np.ascontiguousarray(b)
    assert a.shape == b.shape and a.tobytes() == b.tobytes(), "%s differs" % what


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("gdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("wd", [0.0, 0.1])
def test_bit_exact_over_steps(kind, gdtype, wd):
    ps, gs, ms, dp, dg, plan = _case(SIZES, kind, gdtype, 700)
    for t in (1, 2, 3):
        fq.fp8q_adamw_multi_step(plan, dg, step=t, weight_decay=wd, **HP)
        for i in range(len(SIZES)):
            ps[i], ms[i] = _oracle_step(ps[i], gs[i], ms[i], kind, wd, t)
            _same(host(dp[i]), ps[i], "step %d p[%d]" % (t, i))
            for a, b in zip(_parts(plan, i), ms[i]):
                _same(host(a), b, "step %d moments[%d]" % (t, i))


@pytest.mark.parametrize("kind", KINDS)
def test_late_step_many_tensors_in_several_launches(kind):
    sizes = [1 + (i * 37) % 300 for i in range(450)] + [9000]
    ps, gs, ms, dp, dg, plan = _case(sizes, kind, torch.bfloat16, 900)
    fq.fp8q_adamw_multi_step(plan, dg, step=5000, weight_decay=0.01, **HP)
    for i in range(len(sizes)):
        p, m = _oracle_step(ps[i], gs[i], ms[i], kind, 0.01, 5000)
        _same(host(dp[i]), p, "p[%d]" % i)
        for a, b in zip(_parts(plan, i), m):
            _same(host(a), b, "moments[%d]" % i)


def test_same_as_the_one_tensor_step():
    n = 100003
    ps, gs, ms, dp, dg, plan = _case([n, 300], fq.STATE_E4M3, torch.float32, 40)
    one = [torch.from_numpy(ps[0].copy()).to(DEV), [t.clone() for t in _parts(plan, 0)]]
    fq.fp8q_adamw_multi_step(plan, dg, step=7, weight_decay=0.1, **HP)
    fq.fp8_adam_step(one[0], dg[0], tuple(one[1]), step=7, weight_decay=0.1, **HP)
    assert torch.equal(dp[0], one[0])
    for a, b in zip(_parts(plan, 0), one[1]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("gdtype", [torch.float32, torch.bfloat16])
def test_against_64_bits(gdtype):
    """fp32 moments against the formulas in 64 bits.  m: the coefficients (1 U each), two products and a sum; v: one
    product more; p: the decay, the sqrt, two divisions, a sum, a product and the last difference."""
    sizes, t, wd = [5000, 77, 1], 11, 0.1
    ps, gs, ms, dp, dg, plan = _case(sizes, fq.STATE_F32, gdtype, 60)
    fq.fp8q_adamw_multi_step(plan, dg, step=t, weight_decay=wd, **HP)
    lr, b1, b2, eps = HP["lr"], HP["beta1"], HP["beta2"], HP["eps"]
    for i in range(len(sizes)):
        p, g = ps[i].astype(np.float64), gs[i].astype(np.float64)
        m0, v0 = (a.astype(np.float64) for a in ms[i])
        m = b1 * m0 + (1 - b1) * g
        v = b2 * v0 + (1 - b2) * g * g
        upd = lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps)
        want = p * (1 - lr * wd) - upd
        e_m = 3 * U * (np.abs(b1 * m0) + np.abs((1 - b1) * g)) + 1e-44
        e_v = 5 * U * (np.abs(b2 * v0) + (1 - b2) * g * g) + 1e-44
        # upd: m's error, v's through the root (half), and ten roundings
        e_u = np.abs(upd) * (e_v / np.maximum(v, 1e-300) / 2 + 12 * U) + \
            lr / (1 - b1 ** t) * e_m / (np.sqrt(v / (1 - b2 ** t)) + eps)
        e_p = 3 * U * np.abs(p) + e_u + U * (np.abs(want) + np.abs(upd))
        gm, gv = (host(a).astype(np.float64) for a in _parts(plan, i))
        assert (np.abs(gm - m) <= e_m).all() and (np.abs(gv - v) <= e_v).all()
        assert (np.abs(host(dp[i]).astype(np.float64) - want) <= e_p).all()


@pytest.mark.parametrize("kind", KINDS)
def test_views_at_odd_addresses_and_surroundings(kind):
    """Parameters and gradients as slices of flat buffers at element addresses: nothing else is written."""
    sizes = [1001, 4099, 130, 1]
    ps, gs, ms, _, _, _ = _case(sizes, kind, torch.float32, 80)
    pbuf = torch.full((sum(sizes) + 64,), -7.0, device=DEV)
    gbuf = torch.full((sum(sizes) + 64,), float("nan"), device=DEV)
    dp, dg, at = [], [], 1
    for p, g in zip(ps, gs):
        dp.append(pbuf[at:at + p.size])
        dg.append(gbuf[at + 2:at + 2 + p.size])
        dp[-1].copy_(torch.from_numpy(p))
        dg[-1].copy_(torch.from_numpy(g))
        at += p.size + 5
    plan = fq.fp8q_adamw_plan(dp, kind)
    pad = [torch.full_like(t, 0x7F if t.dtype == torch.uint8 else float("nan")) for t in plan.moments]
    for t, f in zip(plan.moments, pad):
        if t.dtype == torch.uint8 or kind == fq.STATE_F32:
            t.copy_(f)                 # padding holds NaNs; the live part is set next
    for i in range(len(sizes)):
        _put(plan, i, ms[i])
    fq.fp8q_adamw_multi_step(plan, dg, step=3, weight_decay=0.1, **HP)
    live = torch.zeros_like(pbuf, dtype=torch.bool)
    at = 1
    for i, n in enumerate(sizes):
        p, m = _oracle_step(ps[i], gs[i], ms[i], kind, 0.1, 3)
        _same(host(dp[i]), p, "p[%d]" % i)
        for a, b in zip(_parts(plan, i), m):
            _same(host(a), b, "moments[%d]" % i)
        live[at:at + n] = True
        at += n + 5
    assert (pbuf[~live] == -7.0).all()
    for i, n in enumerate(sizes):      # the padding still holds what it held
        for t in plan.moments:
            if t.numel() == plan.blocks[-1] * 128:
                tail = t[plan.blocks[i] * 128 + n:plan.blocks[i + 1] * 128]
                assert (tail == 0x7F).all() if t.dtype == torch.uint8 else torch.isnan(tail).all()


@pytest.mark.parametrize("kind", KINDS)
def test_parameters_without_gradient_are_left(kind):
    sizes = [300, 5000, 64]
    ps, gs, ms, dp, dg, plan = _case(sizes, kind, torch.bfloat16, 90)
    fq.fp8q_adamw_multi_step(plan, [None, dg[1], None], step=2, weight_decay=0.1, **HP)
    for i in range(3):
        p, m = (ps[i], ms[i]) if i != 1 else _oracle_step(ps[i], gs[i], ms[i], kind, 0.1, 2)
        _same(host(dp[i]), p, "p[%d]" % i)
        for a, b in zip(_parts(plan, i), m):
            _same(host(a), b, "moments[%d]" % i)
    before = [p.clone() for p in dp]
    fq.fp8q_adamw_multi_step(plan, [None] * 3, step=3, weight_decay=0.1, **HP)
    assert all(torch.equal(a, b) for a, b in zip(dp, before))


@pytest.mark.parametrize("kind", KINDS)
def test_other_stream_and_moved_parameters(kind):
    ps, gs, ms, dp, dg, plan = _case([3000, 10], kind, torch.float32, 95)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fq.fp8q_adamw_multi_step(plan, dg, step=2, stream=side, **HP)
    torch.cuda.synchronize()
    for i in range(2):
        p, _ = _oracle_step(ps[i], gs[i], ms[i], kind, 0.0, 2)
        _same(host(dp[i]), p, "p[%d]" % i)
    dp[0].data = dp[0].clone()
    with pytest.raises(ValueError, match="moved"):
        fq.fp8q_adamw_multi_step(plan, dg, step=3, **HP)


@pytest.mark.parametrize("kind", KINDS)
def test_tiny_and_huge_moments(kind):
    """Gradients from 1e-30 to 1e10: E4M3 tiles with scales below the fast quotient's range, v beyond fp16's."""
    n = 128 * 40
    g = (torch.randn(n, generator=torch.Generator().manual_seed(4)) *
         torch.logspace(-30, 10, 40).repeat_interleave(128)).float()
    dp = [torch.zeros(n, device=DEV)]
    plan = fq.fp8q_adamw_plan(dp, kind)
    p = np.zeros(n, np.float32)
    state = tuple(host(a).copy() for a in _parts(plan, 0))
    for t in (1, 2):
        fq.fp8q_adamw_multi_step(plan, [g.to(DEV)], step=t, **HP)
        p, state = _oracle_step(p, g.numpy(), state, kind, 0.0, t)
        _same(host(dp[0]), p, "p")
        for a, b in zip(_parts(plan, 0), state):
            _same(host(a), b, "moments")
