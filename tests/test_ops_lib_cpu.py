"""The C ABI of include/fp8q_ops.h on the host: the library exports what the
header declares, and bad arguments get the documented status before a device
is touched (no kernel is launched by these tests)."""
import ctypes
import os
import re

import pytest

import fp8_precision_quant_amd as fq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8q_ops.h")
L = fq._lib
A16 = 1 << 20          # an aligned stand-in for a device pointer, never dereferenced
ODD = A16 + 1
BIG = 1 << 41


def test_header_and_library_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(\w+)\s*\(", text, flags=re.M))
    assert names == set(fq.OPS_SYMBOLS)
    lib = ctypes.CDLL(fq.LIB_PATH)
    for name in names:
        assert hasattr(lib, name), name


def _call(f, base, **changes):
    args = dict(base)
    for k, v in changes.items():
        assert k in args, k
        args[k] = v
    return f(*args.values())


FWD = dict(x=A16, xd=fq.BF16, rows=4, cols=100, ldx=100, w=A16, b=A16, wd=fq.F32, eps=1e-5, y=A16, ldy=100, mean=A16,
           rstd=A16, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(xd=2), fq.ERR_UNSUPPORTED), (dict(wd=-1), fq.ERR_UNSUPPORTED), (dict(eps=-1.0), fq.ERR_UNSUPPORTED),
    (dict(eps=float("nan")), fq.ERR_UNSUPPORTED), (dict(eps=float("inf")), fq.ERR_UNSUPPORTED),
    (dict(rows=-1), fq.ERR_SHAPE), (dict(cols=-1), fq.ERR_SHAPE), (dict(cols=0), fq.ERR_SHAPE),
    (dict(ldx=99), fq.ERR_SHAPE), (dict(ldy=99), fq.ERR_SHAPE), (dict(rows=BIG), fq.ERR_SHAPE),
    (dict(cols=BIG, ldx=BIG, ldy=BIG), fq.ERR_SHAPE), (dict(x=None), fq.ERR_NULL), (dict(y=None), fq.ERR_NULL),
    (dict(x=ODD), fq.ERR_ALIGN), (dict(y=ODD), fq.ERR_ALIGN), (dict(w=A16 + 2), fq.ERR_ALIGN),
    (dict(b=A16 + 2), fq.ERR_ALIGN), (dict(mean=A16 + 2), fq.ERR_ALIGN), (dict(rstd=ODD), fq.ERR_ALIGN),
    (dict(rows=0, x=None, y=None), fq.OK)])
def test_layer_norm_forward_status(change, status):
    assert _call(L.fp8q_layer_norm_forward, FWD, **change) == status


BWD = dict(dy=A16, lddy=100, x=A16, xd=fq.F32, rows=4, cols=100, ldx=100, mean=A16, rstd=A16, w=A16, wd=fq.BF16,
           dx=A16, lddx=100, dw=A16, db=A16, ws=A16, nws=1 << 40, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(xd=9), fq.ERR_UNSUPPORTED), (dict(wd=9), fq.ERR_UNSUPPORTED), (dict(rows=-4), fq.ERR_SHAPE),
    (dict(cols=-4), fq.ERR_SHAPE), (dict(cols=0), fq.ERR_SHAPE), (dict(ldx=99), fq.ERR_SHAPE),
    (dict(lddy=99), fq.ERR_SHAPE), (dict(lddx=99), fq.ERR_SHAPE), (dict(x=None), fq.ERR_NULL),
    (dict(dy=None), fq.ERR_NULL), (dict(mean=None), fq.ERR_NULL), (dict(rstd=None), fq.ERR_NULL),
    (dict(ws=None), fq.ERR_NULL), (dict(nws=16), fq.ERR_SHAPE), (dict(ws=A16 + 4), fq.ERR_ALIGN),
    (dict(x=A16 + 2), fq.ERR_ALIGN), (dict(dy=ODD), fq.ERR_ALIGN), (dict(dx=A16 + 2), fq.ERR_ALIGN),
    (dict(dw=ODD), fq.ERR_ALIGN), (dict(db=ODD), fq.ERR_ALIGN), (dict(w=ODD), fq.ERR_ALIGN),
    (dict(mean=ODD), fq.ERR_ALIGN), (dict(dx=None, dw=None, db=None), fq.OK), (dict(rows=0, cols=0), fq.OK),
    (dict(rows=0, dw=None, db=None), fq.OK)])
def test_layer_norm_backward_status(change, status):
    assert _call(L.fp8q_layer_norm_backward, BWD, **change) == status


def test_workspace_sizes():
    f = L.fp8q_layer_norm_backward_workspace
    assert f(-1, 4) == 0 and f(4, -1) == 0 and f(BIG, 4) == 0
    for rows in (0, 1, 5, 1000, 1 << 20):
        for cols in (1, 100, 4096, 100000):
            assert 0 < f(rows, cols) <= 2048 * 8 * (cols + 16)
    g = L.fp8q_int8_gemm_workspace
    assert g(0, 5, 5) == 0 and g(5, 0, 5) == 0 and g(5, 5, 0) == 0 and g(-1, 5, 5) == 0 and g(4, 4, 1 << 20) == 0
    for M in (1, 16, 96, 333, 4096, 100000):
        for N in (1, 1001, 14336):
            for K in (1, 2049, 14336, 131071):
                assert 0 <= g(M, N, K) <= 64 << 20, (M, N, K)


def _sizes(*n):
    return (ctypes.c_int64 * max(len(n), 1))(*n), len(n)


def test_adamw_table():
    arr, count = _sizes(5, 0, 4096, 4097)
    nbytes = L.fp8q_adamw_table_bytes(count, arr)
    buf = (ctypes.c_int64 * (nbytes // 8 + 1))()
    at = ctypes.addressof(buf)
    assert L.fp8q_adamw_table_fill(count, arr, at, nbytes) == fq.OK
    assert L.fp8q_adamw_table_fill(count, arr, at, nbytes - 8) == fq.ERR_SHAPE
    assert L.fp8q_adamw_table_fill(count, arr, None, nbytes) == fq.ERR_NULL
    assert L.fp8q_adamw_table_fill(count, arr, at + 4, nbytes) == fq.ERR_ALIGN
    header, tensors = list(buf[:4]), [list(buf[4 + 4 * i:8 + 4 * i]) for i in range(count)]
    assert header[1:] == [4, 4, nbytes]
    assert [t[:3] for t in tensors] == [[5, 0, 0], [0, 1, 1], [4096, 1, 1], [4097, 33, 2]]
    chunks = (ctypes.c_uint32 * 8).from_address(at + 32 + 32 * count)
    assert list(chunks) == [0, 0, 2, 0, 3, 0, 3, 32]
    assert L.fp8q_adamw_table_bytes(-1, arr) == -1 and L.fp8q_adamw_table_bytes(2, None) == -1
    for bad in (_sizes(3, -1), _sizes(1 << 41), _sizes(1 << 39)):
        assert L.fp8q_adamw_table_bytes(bad[1], bad[0]) == -1
    assert L.fp8q_adamw_table_bytes(0, None) == 32


def _step_args():
    arr, count = _sizes(5, 0, 300)
    nbytes = L.fp8q_adamw_table_bytes(count, arr)
    table = (ctypes.c_int64 * (nbytes // 8))()
    assert L.fp8q_adamw_table_fill(count, arr, ctypes.addressof(table), nbytes) == fq.OK
    ptr = ctypes.c_void_p * count
    p, g = ptr(A16, None, A16), ptr(A16, None, A16)
    keep = (table, p, g)
    return dict(host=ctypes.addressof(table), dev=A16, p=p, g=g, gd=fq.F32, kind=fq.STATE_E4M3, m=A16, ms=A16, v=A16,
                vs=A16, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, step=1, stream=None), keep


@pytest.mark.parametrize("change,status", [
    (dict(gd=5), fq.ERR_UNSUPPORTED), (dict(kind=2), fq.ERR_UNSUPPORTED), (dict(b1=1.0), fq.ERR_UNSUPPORTED),
    (dict(b2=-0.1), fq.ERR_UNSUPPORTED), (dict(step=0), fq.ERR_UNSUPPORTED), (dict(lr=float("nan")), fq.ERR_UNSUPPORTED),
    (dict(eps=float("inf")), fq.ERR_UNSUPPORTED), (dict(wd=float("nan")), fq.ERR_UNSUPPORTED),
    (dict(host=None), fq.ERR_NULL), (dict(dev=None), fq.ERR_NULL), (dict(p=None), fq.ERR_NULL),
    (dict(g=None), fq.ERR_NULL), (dict(m=None), fq.ERR_NULL), (dict(v=None), fq.ERR_NULL), (dict(ms=None), fq.ERR_NULL),
    (dict(vs=None), fq.ERR_NULL), (dict(m=A16 + 8), fq.ERR_ALIGN), (dict(v=ODD), fq.ERR_ALIGN),
    (dict(ms=ODD), fq.ERR_ALIGN), (dict(vs=A16 + 2), fq.ERR_ALIGN), (dict(dev=A16 + 4), fq.ERR_ALIGN)])
def test_adamw_status(change, status):
    base, keep = _step_args()
    assert _call(L.fp8q_adamw_multi_step, base, **change) == status


def test_adamw_pointer_status():
    base, keep = _step_args()
    ptr = ctypes.c_void_p * 3
    assert _call(L.fp8q_adamw_multi_step, base, p=ptr(None, None, A16)) == fq.ERR_NULL
    assert _call(L.fp8q_adamw_multi_step, base, p=ptr(A16, None, A16 + 2)) == fq.ERR_ALIGN
    assert _call(L.fp8q_adamw_multi_step, base, g=ptr(A16, None, A16 + 2)) == fq.ERR_ALIGN
    assert _call(L.fp8q_adamw_multi_step, base, g=ptr(A16, None, ODD), gd=fq.BF16) == fq.ERR_ALIGN
    junk = (ctypes.c_int64 * 4)(1, 2, 3, 4)
    assert _call(L.fp8q_adamw_multi_step, base, host=ctypes.addressof(junk)) == fq.ERR_SHAPE
    arr, count = _sizes(0, 0)
    table = (ctypes.c_int64 * 12)()
    assert L.fp8q_adamw_table_fill(count, arr, ctypes.addressof(table), 96) == fq.OK
    assert _call(L.fp8q_adamw_multi_step, base, host=ctypes.addressof(table)) == fq.OK     # nothing to step


QUANT = dict(x=A16, xd=fq.BF16, rows=4, cols=100, ldx=100, q=A16, ldq=112, s=A16, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(xd=3), fq.ERR_UNSUPPORTED), (dict(rows=-1), fq.ERR_SHAPE), (dict(cols=-1), fq.ERR_SHAPE),
    (dict(ldx=99), fq.ERR_SHAPE), (dict(ldq=96), fq.ERR_SHAPE), (dict(rows=BIG), fq.ERR_SHAPE),
    (dict(x=None), fq.ERR_NULL), (dict(q=None), fq.ERR_NULL), (dict(s=None), fq.ERR_NULL),
    (dict(cols=0, s=None), fq.ERR_NULL), (dict(x=ODD), fq.ERR_ALIGN), (dict(q=A16 + 8), fq.ERR_ALIGN),
    (dict(ldq=104), fq.ERR_ALIGN), (dict(s=ODD), fq.ERR_ALIGN), (dict(rows=0, s=None), fq.OK)])
def test_quantizer_status(change, status):
    assert _call(L.fp8q_int8_quant_rows, QUANT, **change) == status


GEMM = dict(M=4, N=100, K=200, a=A16, lda=208, sa=A16, b=A16, ldb=208, sb=A16, bias=A16, c=A16, ldc=104, cd=fq.BF16,
            ws=A16, nws=1 << 40, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(cd=4), fq.ERR_UNSUPPORTED), (dict(M=-1), fq.ERR_SHAPE), (dict(N=-1), fq.ERR_SHAPE), (dict(K=-1), fq.ERR_SHAPE),
    (dict(M=BIG), fq.ERR_SHAPE), (dict(K=131072, lda=131072, ldb=131072), fq.ERR_UNSUPPORTED),
    (dict(lda=192), fq.ERR_SHAPE), (dict(ldb=192), fq.ERR_SHAPE), (dict(ldc=96), fq.ERR_SHAPE),
    (dict(lda=1 << 23), fq.ERR_UNSUPPORTED), (dict(ldb=1 << 23), fq.ERR_UNSUPPORTED), (dict(a=None), fq.ERR_NULL),
    (dict(b=None), fq.ERR_NULL), (dict(sa=None), fq.ERR_NULL), (dict(sb=None), fq.ERR_NULL), (dict(c=None), fq.ERR_NULL),
    (dict(K=0, a=None, b=None, sa=None, sb=None, c=None), fq.ERR_NULL), (dict(a=A16 + 8), fq.ERR_ALIGN),
    (dict(b=ODD), fq.ERR_ALIGN), (dict(c=A16 + 2), fq.ERR_ALIGN), (dict(lda=216), fq.ERR_ALIGN),
    (dict(ldb=204), fq.ERR_ALIGN), (dict(ldc=100), fq.ERR_ALIGN), (dict(bias=ODD), fq.ERR_ALIGN),
    (dict(sa=ODD), fq.ERR_ALIGN), (dict(sb=ODD), fq.ERR_ALIGN), (dict(ws=A16 + 4), fq.ERR_ALIGN),
    (dict(M=0, c=None), fq.OK), (dict(N=0, c=None), fq.OK)])
def test_product_status(change, status):
    assert _call(L.fp8q_int8_gemm, GEMM, **change) == status


def test_product_workspace_status():
    """Where the product asks for scratch memory it insists on it."""
    need = L.fp8q_int8_gemm_workspace
    for M in (1, 16, 96, 333):
        size = dict(M=M, N=4096, K=14336, lda=14336, ldb=14336, ldc=4096)
        if need(M, 4096, 14336) > 0:
            assert _call(L.fp8q_int8_gemm, GEMM, ws=None, **size) == fq.ERR_NULL
            assert _call(L.fp8q_int8_gemm, GEMM, nws=need(M, 4096, 14336) - 1, **size) == fq.ERR_SHAPE
