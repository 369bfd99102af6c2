// Matrix product of int8 codes with a scale per row of A (token) and per row
// of B (output channel), for gfx950.
//
//   C[m][n] = (float)(sum_k A[m][k] B[n][k]) * SA[m] * SB[n] + bias[n]
//
// The sum is exact (int32; K <= 131071 keeps K * 128^2 below 2^31), so its
// order and the way it is split never change the result; it is rounded to
// fp32 once and each fp32 operation after it once, in the order above.
#include "gemm_common.h"
#include "gemm_lds.h"
#include "ops_internal.h"
#include "row_io.h"

namespace fp8q {

namespace {

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

// The finished output of 4 consecutive columns n .. n + 3 of row m.
template <typename C>
__device__ __forceinline__ void store4(const Int8Args& p, int64_t m, int64_t n, v4i acc, float sa)
{
    if (n >= p.N) return;
    C* const out = reinterpret_cast<C*>(p.c) + m * p.ldc + n;
    float f[4];
    const int left = p.N - n < 4 ? (int)(p.N - n) : 4;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t c = r < left ? n + r : n;
        f[r] = scaled(acc[r], sa, p.sb[c], p.bias ? p.bias[c] : 0.0f);
    }
    if (left == 4) {
        if constexpr (sizeof(C) == 2) {
            *reinterpret_cast<uint2*>(out) = make_uint2(bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]));
        } else {
            *reinterpret_cast<float4*>(out) = make_float4(f[0], f[1], f[2], f[3]);
        }
    } else {
#pragma unroll
        for (int r = 0; r < 3; ++r)
            if (r < left) out[r] = narrow<C>(f[r]);
    }
}

// ---------------------------------------------------------------------------
// K == 0: the bias, or zeros
// ---------------------------------------------------------------------------

template <typename C>
__global__ __launch_bounds__(256) void int8_gemm_bias_kernel(Int8Args p)
{
    const int64_t n_total = p.M * p.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n_total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / p.N, n = i % p.N;
        reinterpret_cast<C*>(p.c)[m * p.ldc + n] = narrow<C>(p.bias ? p.bias[n] : 0.0f);
    }
}

// ---------------------------------------------------------------------------
// Few tokens: the weight is read once, straight into registers
// ---------------------------------------------------------------------------

// 16 bytes of a row at k, those at or past `K` zero (k a multiple of 16 and
// the row padded to one, so the load stays inside the row's stride).
__device__ __forceinline__ v4i row16(const int8_t* row, int64_t k, int64_t K)
{
    if (k >= K) return v4i{0, 0, 0, 0};
    const uint4 v = mask_bytes(*reinterpret_cast<const uint4*>(row + k), K - k < 16 ? (int)(K - k) : 16);
    return v4i{(int)v.x, (int)v.y, (int)v.z, (int)v.w};
}

// One workgroup makes MB blocks of 16 tokens times 16 output channels; its
// four waves take every fourth 128 bytes of K and meet in LDS at the end, so
// the weight streams through 64-lane loads with U of them in flight, no LDS
// on the way, and nothing is left to join.  Lane l feeds row l % 16 of both
// operands: bytes 32 (l / 16) .. + 31 of the 128, two matrix instructions (any
// pairing of k with lanes will do that is the same for A and B).
template <typename C, int MB>
__global__ __launch_bounds__(256) void int8_gemm_few_kernel(Int8Args p)
{
    constexpr int U = 4;     // 128-byte steps in flight
    __shared__ v4i part[3][MB][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, kg = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t n = n0 + row < p.N ? n0 + row : p.N - 1;     // (rows past N repeat the last: not stored)
    const int8_t* const b = p.b + n * p.ldb;
    const int8_t* a[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) a[i] = p.a + (16 * i + row < p.M ? 16 * i + row : p.M - 1) * p.lda;
    v4i acc[MB] = {};
    const int64_t whole = p.K / 128 * 128;
    int64_t k = (int64_t)wave * 128;
    auto step = [&](const v4i& b0, const v4i& b1, const v4i (&a0)[MB], const v4i (&a1)[MB]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b0, a0[i], acc[i], 0, 0, 0);
            acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b1, a1[i], acc[i], 0, 0, 0);
        }
    };
    for (; k + (U - 1) * 512 < whole; k += U * 512) {
        v4i b0[U], b1[U], a0[U][MB], a1[U][MB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = k + u * 512 + 32 * kg;
            b0[u] = *reinterpret_cast<const v4i*>(b + at);
            b1[u] = *reinterpret_cast<const v4i*>(b + at + 16);
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                a0[u][i] = *reinterpret_cast<const v4i*>(a[i] + at);
                a1[u][i] = *reinterpret_cast<const v4i*>(a[i] + at + 16);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) step(b0[u], b1[u], a0[u], a1[u]);
    }
    for (; k < p.K; k += 512) {
        const int64_t at = k + 32 * kg;
        const v4i b0 = row16(b, at, p.K), b1 = row16(b, at + 16, p.K);
        v4i a0[MB], a1[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            a0[i] = row16(a[i], at, p.K);
            a1[i] = row16(a[i], at + 16, p.K);
        }
        step(b0, b1, a0, a1);
    }
    if (wave > 0)
#pragma unroll
        for (int i = 0; i < MB; ++i) part[wave - 1][i][lane] = acc[i];
    __syncthreads();
    if (wave > 0) return;
    // lane l holds token l % 16 and channels 4 (l / 16) .. + 3
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int64_t m = 16 * i + row;
        const v4i t = acc[i] + part[0][i][lane] + part[1][i][lane] + part[2][i][lane];
        if (m < p.M) store4<C>(p, m, n0 + 4 * kg, t, p.sa[m]);
    }
}

// ---------------------------------------------------------------------------
// Tiles of 128 x BN, staged through LDS; K may be split over workgroups
// ---------------------------------------------------------------------------

constexpr int kBM = 128;
constexpr int kBK = 128;

// Four waves, each 64 x BN / 2 of the tile.  Chunks of 128 along K travel from
// memory to LDS directly, kDepth stages deep, with one barrier per chunk.
// Rows past M or N and bytes past the operand's end read as zero (buffer
// bounds); bytes between K and the next row's start are whatever lies there,
// so the A rows of the last chunk are cleared from K on in LDS, which clears
// the products.  With gridDim.y > 1 workgroup y takes its share of the chunks
// and leaves int32 sums in ws[y][M][nstride] for int8_gemm_join_kernel.
template <typename C, int BN, int DEPTH>
__global__ __launch_bounds__(256) void int8_gemm_tile_kernel(Int8Args p, int tiles_n, int chunks_per, int64_t nstride)
{
    constexpr int NB = BN / 32;               // 16-column blocks per wave
    constexpr int NA = kBM / 32, NL = BN / 32;   // loads of A and B per wave and chunk (8 rows each)
    constexpr int kStage = (kBM + BN) * kBK;
    __shared__ __attribute__((aligned(16))) uint8_t smem[DEPTH * kStage];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * kBM, n0 = (int64_t)(blockIdx.x % tiles_n) * BN;
    const int KB = (int)((p.K + kBK - 1) / kBK);
    const int c0 = blockIdx.y * chunks_per, c1 = min(KB, c0 + chunks_per);
    const int64_t k16 = (p.K + 15) & ~(int64_t)15;
    const int64_t mrows = min(p.M - m0, (int64_t)kBM), nrows = min(p.N - n0, (int64_t)BN);
    const __amdgpu_buffer_rsrc_t ra = rsrc(p.a + m0 * p.lda, (mrows - 1) * p.lda + k16);
    const __amdgpu_buffer_rsrc_t rb = rsrc(p.b + n0 * p.ldb, (nrows - 1) * p.ldb + k16);
    const uint32_t lds0 = lds_addr(smem);
    const int lr = lane >> 3;
    // load t of a wave fills LDS rows 8 (NA wave + t) .. + 7; the slot order within a row depends on the row
    uint32_t va[NA], vb[NL];
#pragma unroll
    for (int t = 0; t < NA; ++t) {
        const int r = 8 * (NA * wave + t) + lr;
        va[t] = (uint32_t)(r * p.lda) + 16u * (uint32_t)((lane & 7) ^ swz_key(r));
    }
#pragma unroll
    for (int t = 0; t < NL; ++t) {
        const int r = 8 * (NL * wave + t) + lr;
        vb[t] = (uint32_t)(r * p.ldb) + 16u * (uint32_t)((lane & 7) ^ swz_key(r));
    }
    auto load = [&](int c, int st) __attribute__((always_inline)) {
        // (past the last chunk: out of bounds, which reads nothing and keeps the count of loads)
        const uint32_t k = c < c1 ? (uint32_t)c * kBK : 0x80000000u;
        const uint32_t base = lds0 + (uint32_t)st * kStage;
#pragma unroll
        for (int t = 0; t < NA; ++t) dma16_at(ra, base + (uint32_t)(8 * (NA * wave + t) * kBK), va[t] + k, 0);
#pragma unroll
        for (int t = 0; t < NL; ++t) dma16_at(rb, base + (uint32_t)((kBM + 8 * (NL * wave + t)) * kBK), vb[t] + k, 0);
    };
    for (int s = 0; s < DEPTH - 1; ++s) load(c0 + s, s);
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * (BN / 2);
    const int row = lane & 15, kg = lane >> 4;
    v4i acc[4][NB] = {};
    int st = 0;
    for (int c = c0; c < c1; ++c) {
        wait_vm<(DEPTH - 2) * (NA + NL)>();      // this wave's loads of chunk c have landed
        uint8_t* const stage = smem + st * kStage;
        if (c == KB - 1 && p.K % kBK) {
            const int valid = (int)(p.K % kBK);
            for (int i = lane; i < 8 * NA * 8; i += 64) {
                const int r = 8 * NA * wave + i / 8, chunk = i % 8;
                if (16 * chunk + 16 > valid) {
                    uint4* const at = reinterpret_cast<uint4*>(stage + sw(r, chunk));
                    *at = mask_bytes(*at, valid > 16 * chunk ? valid - 16 * chunk : 0);
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        __builtin_amdgcn_s_barrier();            // everyone's have, and chunk c - 1 has been read
        const uint32_t base = lds0 + (uint32_t)(st * kStage);
        v4i fa[4][2], fb[NB][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[i][h] = ds128<0>(base + (uint32_t)sw(wm + 16 * i + row, 2 * kg + h));
#pragma unroll
            for (int j = 0; j < NB; ++j) fb[j][h] = ds128<0>(base + (uint32_t)(kBM * kBK + sw(wn + 16 * j + row, 2 * kg + h)));
        }
        load(c + DEPTH - 1, st == 0 ? DEPTH - 1 : st - 1);
        asm volatile("s_waitcnt lgkmcnt(0)"
                     : "+v"(fa[0][0]), "+v"(fa[1][0]), "+v"(fa[2][0]), "+v"(fa[3][0]), "+v"(fa[0][1]), "+v"(fa[1][1]),
                       "+v"(fa[2][1]), "+v"(fa[3][1])
                     :
                     : "memory");
#pragma unroll
        for (int j = 0; j < NB; ++j) asm volatile("" : "+v"(fb[j][0]), "+v"(fb[j][1])::"memory");
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j][h], fa[i][h], acc[i][j], 0, 0, 0);
        st = st == DEPTH - 1 ? 0 : st + 1;
    }
    wait_vm<0>();      // no load may land after the workgroup has ended
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + wm + 16 * i + row;
        if (m >= p.M) continue;
        if (gridDim.y > 1) {
            int32_t* const w = p.ws + ((int64_t)blockIdx.y * p.M + m) * nstride;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int64_t n = n0 + wn + 16 * j + 4 * kg;
                if (n < p.N) *reinterpret_cast<v4i*>(w + n) = acc[i][j];     // (nstride is a multiple of 4)
            }
        } else {
            const float sa = p.sa[m];
#pragma unroll
            for (int j = 0; j < NB; ++j) store4<C>(p, m, n0 + wn + 16 * j + 4 * kg, acc[i][j], sa);
        }
    }
}

// C from the split's sums: four columns a thread.
template <typename C>
__global__ __launch_bounds__(256) void int8_gemm_join_kernel(Int8Args p, int split, int64_t nstride)
{
    const int64_t quads = nstride / 4, total = p.M * quads;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / quads, n = 4 * (i % quads);
        v4i t = {0, 0, 0, 0};
        for (int y = 0; y < split; ++y)
            t += *reinterpret_cast<const v4i*>(p.ws + ((int64_t)y * p.M + m) * nstride + n);
        store4<C>(p, m, n, t, p.sa[m]);
    }
}

// How a product is made, from its sizes alone.
struct Int8Plan {
    int few;             // blocks of 16 tokens of the few-token kernel, or 0
    int bn, split, chunks_per;
    int64_t nstride;
};

Int8Plan int8_plan(int64_t M, int64_t N, int64_t K)
{
    Int8Plan q = {0, 64, 1, 0, (N + 3) / 4 * 4};
    if (M <= 32) {
        q.few = M <= 16 ? 1 : 2;
        return q;
    }
    const int64_t KB = (K + kBK - 1) / kBK, tm = (M + kBM - 1) / kBM;
    if (tm * ((N + 127) / 128) >= 512) q.bn = 128;
    const int64_t tiles = tm * ((N + q.bn - 1) / q.bn);
    int64_t split = tiles >= 256 ? 1 : 512 / tiles;
    if (split > KB / 2) split = KB / 2;
    if (split > 16) split = 16;
    if (split < 1) split = 1;
    q.chunks_per = (int)((KB + split - 1) / split);
    q.split = (int)((KB + q.chunks_per - 1) / q.chunks_per);
    return q;
}

template <typename C, int BN, int DEPTH>
void launch_tile(const Int8Args& p, const Int8Plan& q, hipStream_t st)
{
    const int64_t tiles_n = (p.N + BN - 1) / BN, tiles = (p.M + kBM - 1) / kBM * tiles_n;
    hipLaunchKernelGGL((int8_gemm_tile_kernel<C, BN, DEPTH>), dim3((uint32_t)tiles, (uint32_t)q.split), dim3(256),
                       0, st, p, (int)tiles_n, q.chunks_per, q.nstride);
}

template <typename C>
void launch(const Int8Args& p, hipStream_t st)
{
    if (p.K == 0) {
        const int64_t groups = (p.M * p.N + 255) / 256;
        hipLaunchKernelGGL(int8_gemm_bias_kernel<C>, dim3((uint32_t)(groups < 65536 ? groups : 65536)), dim3(256), 0,
                           st, p);
        return;
    }
    const Int8Plan q = int8_plan(p.M, p.N, p.K);
    if (q.few) {
        const dim3 grid((uint32_t)((p.N + 15) / 16));
        if (q.few == 1) hipLaunchKernelGGL((int8_gemm_few_kernel<C, 1>), grid, dim3(256), 0, st, p);
        else hipLaunchKernelGGL((int8_gemm_few_kernel<C, 2>), grid, dim3(256), 0, st, p);
        return;
    }
    if (q.bn == 128) launch_tile<C, 128, 2>(p, q, st);
    else launch_tile<C, 64, 3>(p, q, st);
    if (q.split > 1) {
        const int64_t groups = (p.M * (q.nstride / 4) + 255) / 256;
        hipLaunchKernelGGL(int8_gemm_join_kernel<C>, dim3((uint32_t)(groups < 65536 ? groups : 65536)), dim3(256), 0,
                           st, p, q.split, q.nstride);
    }
}

}  // namespace

int64_t int8_gemm_workspace(int64_t M, int64_t N, int64_t K)
{
    const Int8Plan q = int8_plan(M, N, K);
    return q.split > 1 ? q.split * M * q.nstride * 4 : 0;
}

void launch_int8_gemm(int64_t M, int64_t N, int64_t K, const int8_t* a, int64_t lda, const float* sa, const int8_t* b,
                      int64_t ldb, const float* sb, const float* bias, void* c, int64_t ldc, int c_dtype, int32_t* ws,
                      hipStream_t st)
{
    const Int8Args p = {M, N, K, a, lda, sa, b, ldb, sb, bias, c, ldc, ws};
    if (c_dtype == FP8Q_BF16) launch<uint16_t>(p, st);
    else launch<float>(p, st);
}

}  // namespace fp8q
