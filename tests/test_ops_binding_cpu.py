"""The argument checks of fp8_precision_quant_amd/operators.py on the host:
every wrapper refuses tensors off the GPU, of another type or shape, with
ValueError and before the library is called (the device check is bypassed and
the library replaced by a stub that fails the test if it is reached)."""
import types

import pytest
import torch

import fp8_precision_quant_amd as fq
from fp8_precision_quant_amd import operators as ops

i8, u8, f32, bf16, f16 = torch.int8, torch.uint8, torch.float32, torch.bfloat16, torch.float16


def z(*shape, dtype=f32):
    return torch.zeros(shape, dtype=dtype)


def test_cpu_tensors_are_rejected():
    x = z(4, 256, dtype=bf16)
    with pytest.raises(ValueError, match="GPU"):
        fq.fp8q_layer_norm_forward(x)
    with pytest.raises(ValueError, match="GPU"):
        fq.fp8q_layer_norm_backward(x, x, z(4), z(4))
    with pytest.raises(ValueError, match="GPU"):
        fq.fp8q_int8_quant_rows(x)
    with pytest.raises(ValueError, match="GPU"):
        fq.fp8q_int8_gemm(z(4, 32, dtype=i8), z(4), z(8, 32, dtype=i8), z(8))
    with pytest.raises(ValueError, match="GPU"):
        fq.fp8q_adamw_plan([z(10)])


class _NoLib:
    def __getattr__(self, name):
        raise AssertionError("the library was called (%s) although the arguments are invalid" % name)


@pytest.fixture
def host(monkeypatch):
    """CPU tensors pass as GPU tensors; the library must not be reached."""
    class Call:
        def __init__(self, first, stream):
            self.dev, self.handle = first.device, 0

        def __call__(self, fn, where, *args):
            raise AssertionError("%s was called although the arguments are invalid" % where)

        def keep(self, *tensors):
            pass
    monkeypatch.setattr(ops, "_Call", Call)
    monkeypatch.setattr(ops, "_device", lambda t, s: t.device)
    monkeypatch.setattr(ops, "_on", lambda dev, **t: None)


def refused(match, f, *args, **kw):
    with pytest.raises(ValueError, match=match):
        f(*args, **kw)


def test_layer_norm_arguments(host):
    x, w, s = z(4, 100, dtype=bf16), z(100), z(4)
    fwd, bwd = fq.fp8q_layer_norm_forward, fq.fp8q_layer_norm_backward
    refused("x must", fwd, z(4, 100, dtype=f16))
    refused("w must be", fwd, x, z(99))
    refused("w must be", fwd, x, z(200)[::2])
    refused("w must be", fwd, x, z(100, dtype=f16))
    refused("b must be", fwd, x, w, z(100, dtype=bf16))       # one type for both
    refused("y must", fwd, x, w, y=z(4, 100))
    refused("y must", fwd, x, w, y=z(5, 100, dtype=bf16))
    refused("mean must", fwd, x, w, mean=z(3))
    refused("rstd must", fwd, x, w, rstd=z(4, dtype=bf16))
    refused("contiguous rows", fwd, z(100, 4, dtype=bf16).t())
    with pytest.raises(ValueError):
        fwd(z(2, 4, 100))
    refused("dy must", bwd, z(4, 100), x, s, s, w)
    refused("dy must", bwd, z(4, 99, dtype=bf16), x, s, s, w)
    refused("dx must", bwd, x, x, s, s, w, dx=z(4, 100))
    refused("mean must", bwd, x, x, z(5), s, w)
    refused("rstd must", bwd, x, x, s, s.to(bf16), w)
    refused("dw must", bwd, x, x, s, s, w, dw=z(100, dtype=bf16))
    refused("db must", bwd, x, x, s, s, w, db=z(101))
    refused("db must", bwd, x, x, s, s, dw=z(100), db=z(100, dtype=bf16))


def test_adamw_arguments(host, monkeypatch):
    plan = fq.fp8q_adamw_plan
    refused("no parameters", plan, [])
    refused("unknown moment state", plan, [z(3)], 7)
    refused("params", plan, [z(3, dtype=bf16)])
    refused("params", plan, [z(4, 4).t()[:, :2]])
    refused("expected 4", plan, [z(3)], fq.STATE_E4M3, (z(128), z(128)))
    refused("moments", plan, [z(3)], fq.STATE_F32, (z(128), z(3)))
    refused("moments", plan, [z(130)], fq.STATE_E4M3, (z(256, dtype=u8), z(2), z(256, dtype=u8), z(1)))
    refused("moments", plan, [z(3)], fq.STATE_E4M3, (z(128), z(1), z(128, dtype=u8), z(1)))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: types.SimpleNamespace(synchronize=lambda: None))
    p = plan([z(3), z(2, 5)], fq.STATE_F32)
    assert p.blocks == [0, 1, 2] and p.sizes == [3, 10] and [t.numel() for t in p.moments] == [256, 256]
    step = fq.fp8q_adamw_multi_step
    refused("plan must", step, None, [], lr=1e-3)
    refused("gradients for", step, p, [z(3)], lr=1e-3)
    refused("grads", step, p, [z(3), z(11)], lr=1e-3)
    refused("grads", step, p, [z(3), z(5, 4).t()[:2]], lr=1e-3)
    refused("grads", step, p, [z(3, dtype=f16), z(10)], lr=1e-3)
    refused("one type", step, p, [z(3), z(10, dtype=bf16)], lr=1e-3)
    assert step(p, [None, None], lr=1e-3) is None
    p.params[0].data = z(3) + 1
    refused("moved", step, p, [z(3), z(10)], lr=1e-3)


def test_int8_arguments(host):
    quant, gemm = fq.fp8q_int8_quant_rows, fq.fp8q_int8_gemm
    refused("x must", quant, z(4, 64, dtype=f16))
    refused("q must", quant, z(4, 64), q=z(4, 64, dtype=u8))
    refused("q must", quant, z(4, 64), q=z(4, 63, dtype=i8))
    refused("s must", quant, z(4, 64), s=z(5))
    refused("contiguous rows", quant, z(64, 4).t())
    a, b, sa, sb = z(4, 32, dtype=i8), z(8, 32, dtype=i8), z(4), z(8)
    refused("contraction", gemm, a, sa, z(8, 48, dtype=i8), sb)
    refused("a must", gemm, z(4, 32, dtype=u8), sa, b, sb)
    refused("b must", gemm, a, sa, z(8, 32, dtype=u8), sb)
    refused("sa must", gemm, a, z(5), b, sb)
    refused("sb must", gemm, a, sa, b, z(16)[::2])
    refused("bias must", gemm, a, sa, b, sb, bias=z(8, dtype=bf16))
    refused("bias must", gemm, a, sa, b, sb, bias=z(9))
    refused("output dtype", gemm, a, sa, b, sb, out_dtype=f16)
    refused("c must", gemm, a, sa, b, sb, c=z(4, 8, dtype=f16))
    refused("c must", gemm, a, sa, b, sb, c=z(4, 9))
    refused("contiguous rows", gemm, z(32, 4, dtype=i8).t(), sa, b, sb)
