// Per-row int8 quantizer for gfx950.
//
//   s = max_c |x| / 127 (IEEE fp32 division),  q = rint(RN_fp32(x / s)), ties
//   to even, saturated to [-127, 127];  s == 0 gives q = 0.
#include "ops_internal.h"
#include "row_io.h"

namespace fp8q {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxRowGroups = (int64_t)1 << 23;
constexpr float kInt8Max = 127.0f;

__device__ __forceinline__ int8_t code(float x, float s)
{
    if (s == 0.0f) return 0;
    return (int8_t)__builtin_amdgcn_fmed3f(__builtin_rintf(x / s), -kInt8Max, kInt8Max);
}

// code(x, s) for a row with s >= 2^-90 (or s = 0 with y = 0): RN(x / s) as a
// corrected reciprocal quotient (q0 = RN(x y), y = RN(1 / s), the residual
// q0 s - x exact, RN(q0 - e y) the rounded quotient: Markstein's theorem),
// |q| <= 127 (1 + 2^-23), then rounded to an integer, ties to even, by the
// addition of 1.5 * 2^23, whose sum's low byte is the code.
__device__ __forceinline__ uint32_t code_bits(float x, float s, float y)
{
    const float q0 = x * y;
    const float e = __builtin_fmaf(q0, s, -x);
    const float q = __builtin_fmaf(-e, y, q0);
    return __float_as_uint(q + 12582912.0f);
}

// bytes 0 of a, b, c, d
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400), __builtin_amdgcn_perm(b, a, 0x0c0c0400),
                                 0x05040100);
}

// Rows of up to TPR * NV vectors of 16 bytes, held in the registers of TPR
// threads between the maximum and the codes.  Vector i starts at element
// min(i kVec, cols - kVec): the last one overlaps its neighbour (repeated
// elements change no maximum and get the same code twice), so every access is
// whole.  Needs cols >= kVec.
template <typename T, int TPR, int NV>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void int8_rows_reg_kernel(const T* __restrict__ x, int64_t rows,
                                                                              int64_t cols, int64_t ldx,
                                                                              int8_t* __restrict__ q, int64_t ldq,
                                                                              float* __restrict__ s)
{
    constexpr int K = kVec<T>;
    constexpr int RPG = TPR == 64 ? 4 : 1;
    typedef uint32_t u32_any __attribute__((aligned(1)));
    __shared__ float red[TPR / 64];
    const int tid = TPR == 64 ? threadIdx.x & 63 : threadIdx.x;
    for (int64_t r = (int64_t)blockIdx.x * RPG + (TPR == 64 ? threadIdx.x >> 6 : 0); r < rows;
         r += (int64_t)gridDim.x * RPG) {
        const T* xr = x + r * ldx;
        u32x4 raw[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * TPR + tid) * K;
            raw[k] = load16(xr + (c <= cols - K ? c : cols - K));
        }
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float v[K];
            unpack<T>(raw[k], v);
#pragma unroll
            for (int i = 0; i < K; ++i) m = fmaxf(m, fabsf(v[i]));
        }
        m = wave_max(m);
        if constexpr (TPR > 64) {
            __syncthreads();   // the previous row's reads are over
            if ((tid & 63) == 0) red[tid >> 6] = m;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < TPR / 64; ++k) m = fmaxf(m, red[k]);
        }
        const float sc = m / kInt8Max;
        if (tid == 0) s[r] = sc;
        const bool exact = sc != 0.0f && !(sc >= kFastScaleMin);   // the plain quotient
        const float yr = sc == 0.0f || exact ? 0.0f : 1.0f / sc;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * TPR + tid) * K;
            if (c >= cols) continue;
            float v[K];
            uint32_t w[K];
            unpack<T>(raw[k], v);
            if (exact) {
#pragma unroll
                for (int i = 0; i < K; ++i) w[i] = (uint32_t)(int)code(v[i], sc);
            } else {
#pragma unroll
                for (int i = 0; i < K; ++i) w[i] = code_bits(v[i], sc, yr);
            }
            u32_any* out = reinterpret_cast<u32_any*>(q + r * ldq + (c <= cols - K ? c : cols - K));
#pragma unroll
            for (int h = 0; h < K / 4; ++h) out[h] = bytes4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
        }
    }
}

// Rows of any length: one workgroup per row, the row read twice.
template <typename T>
__global__ __launch_bounds__(kThreads) void int8_rows_kernel(const T* __restrict__ x, int64_t rows, int64_t cols,
                                                             int64_t ldx, int8_t* __restrict__ q, int64_t ldq,
                                                             float* __restrict__ s)
{
    __shared__ float red[kThreads / 64];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        float m = 0.0f;
        for (int64_t c = threadIdx.x; c < cols; c += kThreads) m = fmaxf(m, fabsf(widen(x[r * ldx + c])));
        m = wave_max(m);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
        __syncthreads();
        for (int k = 0; k < kThreads / 64; ++k) m = fmaxf(m, red[k]);
        const float sc = m / kInt8Max;
        for (int64_t c = threadIdx.x; c < cols; c += kThreads) q[r * ldq + c] = code(widen(x[r * ldx + c]), sc);
        if (threadIdx.x == 0) s[r] = sc;
    }
}

template <typename T, int TPR, int NV>
void quant_rows(const void* x, int64_t rows, int64_t cols, int64_t ldx, int8_t* q, int64_t ldq, float* s,
                hipStream_t st)
{
    constexpr int threads = TPR > 256 ? TPR : 256;
    constexpr int rpg = TPR == 64 ? 4 : 1;
    const int64_t groups = (rows + rpg - 1) / rpg, most = kMaxRowGroups / (threads / 256);
    hipLaunchKernelGGL((int8_rows_reg_kernel<T, TPR, NV>), dim3((uint32_t)(groups < most ? groups : most)),
                       dim3(threads), 0, st, (const T*)x, rows, cols, ldx, q, ldq, s);
}

template <typename T>
void quant(const void* x, int64_t rows, int64_t cols, int64_t ldx, int8_t* q, int64_t ldq, float* s, hipStream_t st)
{
    const int64_t V = (cols + kVec<T> - 1) / kVec<T>;
    if (cols >= kVec<T>) {
        if (V <= 64) return quant_rows<T, 64, 1>(x, rows, cols, ldx, q, ldq, s, st);
        if (V <= 128) return quant_rows<T, 64, 2>(x, rows, cols, ldx, q, ldq, s, st);
        if (V <= 256) return quant_rows<T, 256, 1>(x, rows, cols, ldx, q, ldq, s, st);
        if (V <= 512) return quant_rows<T, 256, 2>(x, rows, cols, ldx, q, ldq, s, st);
        if (V <= 1024) return quant_rows<T, 256, 4>(x, rows, cols, ldx, q, ldq, s, st);
        if (V <= 2048) return quant_rows<T, 256, 8>(x, rows, cols, ldx, q, ldq, s, st);
        if (V <= 8192) return quant_rows<T, 1024, 8>(x, rows, cols, ldx, q, ldq, s, st);
    }
    const dim3 grid((uint32_t)(rows < kMaxRowGroups ? rows : kMaxRowGroups));
    hipLaunchKernelGGL(int8_rows_kernel<T>, grid, dim3(kThreads), 0, st, (const T*)x, rows, cols, ldx, q, ldq, s);
}

}  // namespace

void launch_int8_quant_rows(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, int8_t* q,
                            int64_t ldq, float* s, hipStream_t st)
{
    if (x_dtype == FP8Q_BF16) quant<uint16_t>(x, rows, cols, ldx, q, ldq, s, st);
    else quant<float>(x, rows, cols, ldx, q, ldq, s, st);
}

}  // namespace fp8q
