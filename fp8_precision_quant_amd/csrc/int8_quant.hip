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

// One workgroup per row, the row read twice.
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

}  // namespace

void launch_int8_quant_rows(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, int8_t* q,
                            int64_t ldq, float* s, hipStream_t st)
{
    const dim3 grid((uint32_t)(rows < kMaxRowGroups ? rows : kMaxRowGroups));
    if (x_dtype == FP8Q_BF16)
        hipLaunchKernelGGL(int8_rows_kernel<uint16_t>, grid, dim3(kThreads), 0, st, (const uint16_t*)x, rows, cols,
                           ldx, q, ldq, s);
    else
        hipLaunchKernelGGL(int8_rows_kernel<float>, grid, dim3(kThreads), 0, st, (const float*)x, rows, cols, ldx, q,
                           ldq, s);
}

}  // namespace fp8q
