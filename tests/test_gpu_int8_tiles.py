"""The int8 product at sizes that take each of its tiles, splits and pairs of
launches, with rows, columns and K that end inside a tile.  The sum is exact,
so every way of making it gives the same bits: the result is compared with
the 64-bit one within the fp32 roundings that follow the sum, and codes past
K, rows past M and columns past N hold values that must not matter."""
import pytest
import torch

import fp8_precision_quant_amd as fq
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
bf16, f32 = torch.bfloat16, torch.float32

# (M, N, K): the tile of 256 x 256; 128 x 256; 128 x 128, whole and K in three; 64 x 128, whole and K in three;
# 64 x 64, whole and K split 4 to 16 ways; rounds of 256 x 256 with 128 x 256, 64 x 128 and 64 x 64 beside them;
# K of one chunk, of fewer bytes than a step and of a whole number of chunks; few tokens, 8 and 16 waves
SIZES = [(1290, 9400, 650), (2005, 4090, 2001), (1023, 4095, 1001), (2208, 508, 10293), (2050, 9000, 520),
         (411, 2958, 12801), (333, 1001, 2049), (129, 1000, 4000), (118, 70, 8192), (33, 48, 20000),
         (4096, 14336, 900), (3990, 9001, 700), (2000, 9000, 1030), (1290, 9400, 100), (1290, 9400, 40),
         (1290, 9400, 256), (2005, 4090, 128), (70, 200, 65), (9, 130, 300000 // 16), (16, 14336, 2000),
         (5, 4096, 9001), (20, 200, 9000)]


def _codes(rows, cols, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    buf = torch.full((rows, -(-cols // 16) * 16), 119, dtype=torch.int8, device=DEV)
    buf[:, :cols] = torch.randint(-127, 128, (rows, cols), generator=g, device=DEV, dtype=torch.int8)
    return buf[:, :cols]


@pytest.mark.parametrize("bias,out", [(False, bf16), (True, f32), (True, bf16)])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_every_tile(M, N, K, bias, out):
    print("int8 product", M, N, K, bias, out, flush=True)
    a, b = _codes(M, K, 1), _codes(N, K, 2)
    g = torch.Generator(device=DEV).manual_seed(3)
    sa, sb = (torch.rand(n, generator=g, device=DEV) * 0.01 + 1e-4 for n in (M, N))
    bs = torch.randn(N, generator=g, device=DEV) if bias else None
    c = fq.fp8q_int8_gemm(a, sa, b, sb, bias=bs, out_dtype=out)
    again = fq.fp8q_int8_gemm(a, sa, b, sb, bias=bs, out_dtype=out)
    assert torch.equal(c, again)
    t = (a.double() @ b.double().t().contiguous()).mul_(sa.double()[:, None]).mul_(sb.double())   # the sum exact
    want = t if bs is None else t + bs.double()
    # the conversion and two products, U each, the bias's sum, then the output's half step
    tol = 1.01 * (3 * U * t.abs() + (0 if bs is None else U * want.abs())) + torch.finfo(out).eps / 2 * want.abs() * 1.01
    bad = ~((c.double() - want).abs() <= tol + 1e-37)
    assert not bad.any(), "%d off, first at %s" % (int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("M,N,K", [(1290, 9400, 650), (2000, 9000, 1030), (2208, 508, 3000)])
def test_nothing_outside_the_output_is_written(M, N, K):
    a, b = _codes(M, K, 5), _codes(N, K, 6)
    one = lambda n: torch.ones(n, device=DEV)
    ld = -(-N // 8) * 8 + 24
    buf = torch.full((M + 2, ld), 77.0, dtype=bf16, device=DEV)
    c = fq.fp8q_int8_gemm(a, one(M), b, one(N), c=buf[1:M + 1, 8:8 + N])
    assert torch.equal(c, fq.fp8q_int8_gemm(a, one(M), b, one(N)))
    outside = buf.clone()
    outside[1:M + 1, 8:8 + N] = 77.0
    assert (outside == 77.0).all()
