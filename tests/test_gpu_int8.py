"""The per-row int8 quantizer and the int8 product on the GPU.

The quantizer's scale and codes are defined to the bit (IEEE division, ties to
even) and compared so, against numpy in fp32 (whose division and rint are
those) and in 64 bits.  The product's sum is exact: the result is compared
with 64-bit integers, within the fp32 roundings that follow the sum: the
conversion, two products and the bias, U = 2^-24 each, then the output's.
"""
import numpy as np
import pytest
import torch

import fp8_precision_quant_amd as fq
from gpu_util import DEV, host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
bf16, f32 = torch.bfloat16, torch.float32


def _rows(rows, cols, seed, dtype):
    x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed))
    x = x * torch.exp(torch.randn(rows, 1, generator=torch.Generator().manual_seed(seed + 1)))
    return x.to(dtype)


def quant_ref(x):
    """Codes and scales of a host tensor in fp32 (numpy's division is IEEE's)."""
    x = x.float().numpy()
    s = (np.abs(x).max(axis=1) if x.shape[1] else np.zeros(x.shape[0], np.float32)) / np.float32(127)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(x / s[:, None])
    return np.clip(np.where(s[:, None] > 0, q, 0), -127, 127).astype(np.int8), s.astype(np.float32)


QSHAPES = [(1, 1), (1, 15), (2, 16), (3, 17), (5, 100), (1, 511), (4, 512), (3, 513), (2, 1000), (7, 2047), (16, 4096),
           (3, 4097), (2, 8191), (5, 8192), (2, 8200), (1, 16384), (2, 16385), (1, 33333), (1, 70000), (1500, 48)]


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("rows,cols", QSHAPES)
def test_quantizer_bits(rows, cols, dtype):
    x = _rows(rows, cols, rows * 7 + cols, dtype)
    q, s = fq.fp8q_int8_quant_rows(x.to(DEV))
    assert q.dtype == torch.int8 and q.stride(0) % 16 == 0
    wq, ws = quant_ref(x)
    assert np.array_equal(host(s).view(np.uint32), ws.view(np.uint32))
    assert np.array_equal(host(q), wq)


def test_quantizer_edges():
    """Zero rows, signed zeros, ties, subnormals, rows whose scale is subnormal or underflows, the largest values."""
    tie = torch.zeros(9, 256)
    tie[1, 5] = -0.0
    tie[2, :] = torch.arange(256) - 128.0            # amax 128: quotients off the integers
    tie[3, :127] = torch.arange(127) + 0.5           # amax 127: s = 1, ties
    tie[3, 200] = -127.0
    tie[4, 7] = 3.4e38
    tie[4, 8] = 1.3e36
    tie[5, :] = torch.randn(256, generator=torch.Generator().manual_seed(1)) * 1e-38
    tie[6, 0:4] = torch.tensor([1e-45, -1e-45, 2.8e-45, 0.0])
    tie[7, :] = torch.randn(256, generator=torch.Generator().manual_seed(2)) * 2e-43
    tie[8, :] = torch.randn(256, generator=torch.Generator().manual_seed(3)) * 1e-30
    q, s = fq.fp8q_int8_quant_rows(tie.to(DEV))
    wq, ws = quant_ref(tie)
    assert np.array_equal(host(s).view(np.uint32), ws.view(np.uint32))
    assert np.array_equal(host(q), wq)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_quantizer_many_quotients(dtype):
    """2^22 quotients of random scales against the IEEE quotient's rounding."""
    x = _rows(1024, 4096, 11, f32) * torch.exp(8 * torch.randn(1024, 1, generator=torch.Generator().manual_seed(5)))
    x = x.to(dtype)
    q, s = fq.fp8q_int8_quant_rows(x.to(DEV))
    wq, ws = quant_ref(x)
    assert np.array_equal(host(s).view(np.uint32), ws.view(np.uint32)) and np.array_equal(host(q), wq)


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("cols,ld,at", [(33, 37, 1), (1000, 1003, 3), (5000, 5001, 1), (17001, 17007, 5)])
def test_quantizer_strides_and_surroundings(cols, ld, at, dtype):
    rows = 4
    x = _rows(rows, cols, 3, dtype)
    buf = torch.full((rows * ld + at + 8,), float("nan"), dtype=dtype, device=DEV)
    view = buf[at:at + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(x)
    pad = -(-cols // 16) * 16 + 16
    qbuf = torch.full((rows + 1, pad), 77, dtype=torch.int8, device=DEV)
    sbuf = torch.full((rows + 2,), -3.0, device=DEV)
    fq.fp8q_int8_quant_rows(view, q=qbuf[:rows, :cols], s=sbuf[1:rows + 1])
    wq, ws = quant_ref(x)
    assert np.array_equal(host(qbuf)[:rows, :cols], wq) and np.array_equal(host(sbuf)[1:rows + 1], ws)
    assert (qbuf[:rows, cols:] == 77).all() and (qbuf[rows] == 77).all()
    assert sbuf[0] == -3.0 and sbuf[rows + 1] == -3.0


def test_quantizer_empty():
    q, s = fq.fp8q_int8_quant_rows(torch.empty(0, 64, device=DEV))
    assert q.shape == (0, 64) and s.numel() == 0
    q, s = fq.fp8q_int8_quant_rows(torch.empty(3, 0, device=DEV))
    assert q.shape == (3, 0) and (s == 0).all()


def _codes(rows, cols, seed, junk=True, top=127):
    """int8 codes on the GPU with rows padded to 16 bytes, the padding full of other values."""
    q = torch.randint(-top, top + 1, (rows, cols), generator=torch.Generator().manual_seed(seed), dtype=torch.int8)
    ld = -(-max(cols, 1) // 16) * 16
    buf = torch.full((rows, ld), 113 if junk else 0, dtype=torch.int8)
    buf[:, :cols] = q
    return q, buf.to(DEV)[:, :cols]


def product_ref(a, b, sa, sb, bias, out):
    """(C, bound) in 64 bits."""
    c = (a.to(DEV).double() @ b.to(DEV).double().t().contiguous())        # exact: below 2^53
    t = c * sa.double()[:, None] * sb.double()
    want = t if bias is None else t + bias.double()
    e = 3 * U * t.abs() + (0 if bias is None else U * want.abs())
    return want, 1.01 * e + torch.finfo(out).eps / 2 * (want.abs() + e) + 1e-37


def _scales(n, seed):
    return torch.exp(torch.randn(n, generator=torch.Generator().manual_seed(seed))).mul(0.01).to(DEV)


def _check_product(M, N, K, bias, out, seed=1, top=127):
    a, da = _codes(M, K, seed, top=top)
    b, db = _codes(N, K, seed + 1, top=top)
    sa, sb = _scales(M, seed + 2), _scales(N, seed + 3)
    bs = torch.randn(N, generator=torch.Generator().manual_seed(seed + 4)).to(DEV) if bias else None
    c = fq.fp8q_int8_gemm(da, sa, db, sb, bias=bs, out_dtype=out)
    assert c.dtype == out and c.shape == (M, N)
    want, tol = product_ref(a, b, sa, sb, bs, out)
    d = (c.double() - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), "%d off, first at %s" % (int(bad.sum()), bad.nonzero()[0].tolist())


GEMMS = [(1, 1, 1), (1, 16, 16), (2, 3, 5), (1, 130, 64), (1, 1000, 129), (3, 257, 1000), (7, 64, 4096), (8, 500, 640),
         (9, 100, 127), (15, 129, 128), (16, 256, 256), (17, 255, 257), (31, 96, 2048), (32, 1024, 96), (33, 200, 500),
         (63, 65, 1025), (64, 64, 64), (65, 1, 2049), (96, 4096, 2048), (100, 33, 4100), (127, 300, 384), (128, 256, 128),
         (129, 257, 1040), (200, 16, 14336), (255, 511, 96), (256, 512, 512), (300, 1024, 2176), (333, 1001, 2049),
         (512, 768, 1024), (1000, 100, 300), (1, 14336, 4096), (4, 4096, 14336), (513, 2050, 1111), (40, 40, 20000)]


@pytest.mark.parametrize("out", [bf16, f32])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M,N,K", GEMMS)
def test_product(M, N, K, bias, out):
    _check_product(M, N, K, bias, out, seed=M + N + K)


@pytest.mark.parametrize("M", [1, 20, 150, 600])
def test_product_largest_sums(M):
    """All codes at the ends of the range, K at its limit: sums near 2^31 stay exact."""
    K, N = 131071, 80
    a = torch.full((M, 131072), -128, dtype=torch.int8, device=DEV)[:, :K]
    b = torch.full((N, 131072), -128, dtype=torch.int8, device=DEV)[:, :K]
    b[1::2] = 127
    one = torch.ones(max(M, N), device=DEV)
    c = fq.fp8q_int8_gemm(a, one[:M], b, one[:N], out_dtype=f32)
    for n, code in ((0, -128), (1, 127)):
        want = np.float32(-128 * code * K)
        assert (c[:, n] == float(want)).all()
        assert (c[:, n::2] == float(want)).all()


def test_product_empty_and_no_k():
    e = torch.empty
    i8 = torch.int8
    one = torch.ones(8, device=DEV)
    c = fq.fp8q_int8_gemm(e(0, 32, dtype=i8, device=DEV), one[:0], e(8, 32, dtype=i8, device=DEV), one)
    assert c.shape == (0, 8)
    a, b = e(3, 16, dtype=i8, device=DEV)[:, :0], e(8, 16, dtype=i8, device=DEV)[:, :0]
    bias = torch.arange(8.0, device=DEV)
    assert torch.equal(fq.fp8q_int8_gemm(a, one[:3], b, one, bias=bias, out_dtype=f32), bias.expand(3, 8))
    assert (fq.fp8q_int8_gemm(a, one[:3] * float("nan"), b, one) == 0).all()


@pytest.mark.parametrize("M,N,K", [(1, 100, 100), (5, 77, 640), (40, 130, 200), (200, 300, 1000), (300, 520, 384)])
@pytest.mark.parametrize("out", [bf16, f32])
def test_product_surroundings_and_strides(M, N, K, out):
    """Operand and output rows inside wider buffers: same bits, nothing outside [0, M) x [0, N) written."""
    a, da = _codes(M, K, 5)
    b, db = _codes(N, K, 6)
    sa, sb = _scales(M, 7), _scales(N, 8)
    plain = fq.fp8q_int8_gemm(da, sa, db, sb, out_dtype=out)
    ld = -(-K // 16) * 16 + 48
    A = torch.full((M + 1, ld), -99, dtype=torch.int8, device=DEV)
    B = torch.full((N + 1, ld), -98, dtype=torch.int8, device=DEV)
    A[:M, :K], B[:N, :K] = a.to(DEV), b.to(DEV)
    C = torch.full((M + 2, -(-N // 8) * 8 + 24), -7.0, dtype=out, device=DEV)
    fq.fp8q_int8_gemm(A[:M, :K], sa, B[:N, :K], sb, c=C[:M, :N])
    assert torch.equal(C[:M, :N], plain)
    assert (C[M:] == -7.0).all() and (C[:, N:] == -7.0).all()


def test_product_non_finite_scales_stay_alone():
    a, da = _codes(20, 300, 1)
    b, db = _codes(50, 300, 2)
    sa, sb = _scales(20, 3), _scales(50, 4)
    clean = fq.fp8q_int8_gemm(da, sa, db, sb)
    sa[3] = float("nan")
    sb[7] = float("inf")
    c = fq.fp8q_int8_gemm(da, sa, db, sb)
    assert torch.isnan(c[3]).all()
    keep = torch.ones_like(c, dtype=torch.bool)
    keep[3], keep[:, 7] = False, False
    assert torch.equal(c[keep], clean[keep])


@pytest.mark.parametrize("M,N,K", [(1, 700, 1000), (48, 300, 4096), (300, 600, 1500)])
def test_product_same_bits_every_time_and_other_stream(M, N, K):
    _, da = _codes(M, K, 1)
    _, db = _codes(N, K, 2)
    sa, sb = _scales(M, 3), _scales(N, 4)
    first = fq.fp8q_int8_gemm(da, sa, db, sb)
    x = _rows(M, K, 9, bf16).to(DEV)
    q0, s0 = fq.fp8q_int8_quant_rows(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        c = fq.fp8q_int8_gemm(da, sa, db, sb, stream=side)
        q, s = fq.fp8q_int8_quant_rows(x, stream=side.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(c, first) and torch.equal(q, q0) and torch.equal(s, s0)


@pytest.mark.parametrize("M", [2, 40, 300])
def test_product_offsets_past_32_bits(M):
    """Operands and output spread over more than 4 GiB by their row strides."""
    K, N, ld = 272, 600, (1 << 23) - 16
    a, b = _codes(M, K, 1)[0], _codes(N, K, 2)[0]
    sa, sb = _scales(M, 3), _scales(N, 4)
    want = fq.fp8q_int8_gemm(a.to(DEV).contiguous(), sa, b.to(DEV).contiguous(), sb)
    B = torch.empty(N, ld, dtype=torch.int8, device=DEV)
    B[:, :K] = b.to(DEV)
    A = torch.empty(M, ld, dtype=torch.int8, device=DEV)
    A[:, :K] = a.to(DEV)
    C = torch.empty(M, (1 << 32) // max(M // 2, 1) // 2 // 8 * 8 + 8, dtype=bf16, device=DEV)
    fq.fp8q_int8_gemm(A[:, :K], sa, B[:, :K], sb, c=C[:, :N])
    assert torch.equal(C[:, :N], want)


def test_quantize_and_multiply():
    """The two together approximate the product of the unquantized operands: each code is off by at most half a
    step, so |error| <= sum_k (|x| sw / 2 + |w| sx / 2 + sx sw / 4)."""
    x = _rows(70, 500, 1, bf16).to(DEV)
    w = _rows(130, 500, 2, bf16).to(DEV)
    (qx, sx), (qw, sw) = fq.fp8q_int8_quant_rows(x), fq.fp8q_int8_quant_rows(w)
    c = fq.fp8q_int8_gemm(qx, sx, qw, sw, out_dtype=f32).double()
    X, W, sx, sw = x.double(), w.double(), sx.double()[:, None], sw.double()
    bound = (X.abs().sum(1, keepdim=True) * sw / 2 + W.abs().sum(1) * sx / 2 + 500 * sx * sw / 4)
    assert ((c - X @ W.t().contiguous()).abs() <= 1.001 * bound).all()
