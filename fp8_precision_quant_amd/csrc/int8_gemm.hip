// Matrix product of int8 codes with a scale per row of A (token) and per row
// of B (output channel), for gfx950.
//
//   C[m][n] = (float)(sum_k A[m][k] B[n][k]) * SA[m] * SB[n] + bias[n]
//
// The sum is exact (int32; K <= 131071 keeps K * 128^2 below 2^31), so its
// order and the way it is split never change the result; it is rounded to
// fp32 once and each fp32 operation after it once, in the order above.
#include "gemm_common.h"
#include "ops_internal.h"
#include "row_io.h"

namespace fp8q {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float scaled(int acc, float sa, float sb, float bias)
{
#pragma clang fp contract(off)
    const float t = (float)acc * sa;
    const float u = t * sb;
    return u + bias;
}

struct Int8Args {
    int64_t M, N, K;
    const int8_t* a;
    int64_t lda;
    const float* sa;
    const int8_t* b;
    int64_t ldb;
    const float* sb;
    const float* bias;
    void* c;
    int64_t ldc;
    int32_t* ws;
};

// 64 x 64 tile, four waves of 32 x 32, chunks of 64 along K staged through
// LDS.  Rows past M or N read the last row (their outputs are not stored);
// bytes past K are zeroed.
constexpr int kSmallTile = 64;

template <typename C>
__global__ __launch_bounds__(256) void int8_gemm_tile64_kernel(Int8Args p)
{
    __shared__ __attribute__((aligned(16))) int8_t sA[kSmallTile][80], sB[kSmallTile][80];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t tiles_n = (p.N + kSmallTile - 1) / kSmallTile;
    const int64_t m0 = (blockIdx.x / tiles_n) * kSmallTile, n0 = (blockIdx.x % tiles_n) * kSmallTile;
    const int lr = tid >> 2, lc = (tid & 3) * 16;
    const int64_t ar = m0 + lr < p.M ? m0 + lr : p.M - 1, br = n0 + lr < p.N ? n0 + lr : p.N - 1;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    v4i acc[2][2] = {};
    for (int64_t k0 = 0; k0 < p.K; k0 += 64) {
        const int64_t left = p.K - (k0 + lc);
        uint4 va = {0, 0, 0, 0}, vb = {0, 0, 0, 0};
        if (left > 0) {
            const int valid = left < 16 ? (int)left : 16;
            va = mask_bytes(*reinterpret_cast<const uint4*>(p.a + ar * p.lda + k0 + lc), valid);
            vb = mask_bytes(*reinterpret_cast<const uint4*>(p.b + br * p.ldb + k0 + lc), valid);
        }
        __syncthreads();
        *reinterpret_cast<uint4*>(&sA[lr][lc]) = va;
        *reinterpret_cast<uint4*>(&sB[lr][lc]) = vb;
        __syncthreads();
        v4i fa[2], fb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            fa[i] = *reinterpret_cast<const v4i*>(&sA[wm + 16 * i + (lane & 15)][(lane >> 4) * 16]);
            fb[i] = *reinterpret_cast<const v4i*>(&sB[wn + 16 * i + (lane & 15)][(lane >> 4) * 16]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
    // lane l holds row m = l % 16 and columns n = 4 (l / 16) .. + 3 of a block
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t m = m0 + wm + 16 * i + (lane & 15);
        if (m >= p.M) continue;
        const float sa = p.K > 0 ? p.sa[m] : 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t n = n0 + wn + 16 * j + 4 * (lane >> 4) + r;
                if (n >= p.N) continue;
                const float sb = p.K > 0 ? p.sb[n] : 0.0f;
                reinterpret_cast<C*>(p.c)[m * p.ldc + n] =
                    narrow<C>(scaled(acc[i][j][r], sa, sb, p.bias ? p.bias[n] : 0.0f));
            }
    }
}

}  // namespace

int64_t int8_gemm_workspace(int64_t, int64_t, int64_t) { return 0; }

void launch_int8_gemm(int64_t M, int64_t N, int64_t K, const int8_t* a, int64_t lda, const float* sa, const int8_t* b,
                      int64_t ldb, const float* sb, const float* bias, void* c, int64_t ldc, int c_dtype, int32_t* ws,
                      hipStream_t st)
{
    const Int8Args p = {M, N, K, a, lda, sa, b, ldb, sb, bias, c, ldc, ws};
    const int64_t tiles = ((M + kSmallTile - 1) / kSmallTile) * ((N + kSmallTile - 1) / kSmallTile);
    if (c_dtype == FP8Q_BF16)
        hipLaunchKernelGGL(int8_gemm_tile64_kernel<uint16_t>, dim3((uint32_t)tiles), dim3(256), 0, st, p);
    else
        hipLaunchKernelGGL(int8_gemm_tile64_kernel<float>, dim3((uint32_t)tiles), dim3(256), 0, st, p);
}

}  // namespace fp8q
