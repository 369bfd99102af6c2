// Layer norm over the last axis, forward and backward, for gfx950.
//
//   mean = sum_c x / C,  var = sum_c (x - mean)^2 / C,  rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,  y = xh w + b
//   u = dy w,  dx = rstd (u - sum_c u / C - xh sum_c (u xh) / C)
//   dw = sum_r dy xh,  db = sum_r dy
//
// All statistics and sums are fp32; each output is rounded once.  Every sum
// has a fixed order (no atomics): the same call gives the same bits.
#include "ops_internal.h"
#include "row_io.h"

namespace fp8q {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
// workgroups of a row-wise launch (the total of threads must fit 32 bits)
constexpr int64_t kMaxRowGroups = (int64_t)1 << 23;

// sums of a workgroup, in every thread (s: kWaves floats per value)
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* s)
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    __syncthreads();   // the previous use of s is over
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) s[i * kWaves + (threadIdx.x >> 6)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) v[i] += s[i * kWaves + k];
    }
}

// One workgroup per row, the row read once per pass.
template <typename T, typename W>
__global__ __launch_bounds__(kThreads) void ln_fwd_kernel(const T* __restrict__ x, int64_t rows, int64_t cols,
                                                          int64_t ldx, const W* __restrict__ w,
                                                          const W* __restrict__ b, float eps, T* __restrict__ y,
                                                          int64_t ldy, float* __restrict__ mean,
                                                          float* __restrict__ rstd)
{
    __shared__ float red[kWaves];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* xr = x + r * ldx;
        float s[1] = {0.0f};
        for (int64_t c = threadIdx.x; c < cols; c += kThreads) s[0] += widen(xr[c]);
        group_sum(s, red);
        const float mu = s[0] / (float)cols;
        s[0] = 0.0f;
        for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
            const float d = widen(xr[c]) - mu;
            s[0] += d * d;
        }
        group_sum(s, red);
        const float rs = 1.0f / __builtin_sqrtf(s[0] / (float)cols + eps);
        for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
            const float xh = (widen(xr[c]) - mu) * rs;
            y[r * ldy + c] = narrow<T>(xh * (w ? widen(w[c]) : 1.0f) + (b ? widen(b[c]) : 0.0f));
        }
        if (threadIdx.x == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

template <typename T, typename W>
__global__ __launch_bounds__(kThreads) void ln_bwd_dx_kernel(const T* __restrict__ dy, int64_t lddy,
                                                             const T* __restrict__ x, int64_t rows, int64_t cols,
                                                             int64_t ldx, const float* __restrict__ mean,
                                                             const float* __restrict__ rstd, const W* __restrict__ w,
                                                             T* __restrict__ dx, int64_t lddx)
{
    __shared__ float red[2 * kWaves];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const float mu = mean[r], rs = rstd[r];
        const T* xr = x + r * ldx;
        const T* gr = dy + r * lddy;
        float s[2] = {0.0f, 0.0f};
        for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
            const float u = widen(gr[c]) * (w ? widen(w[c]) : 1.0f);
            s[0] += u;
            s[1] += u * ((widen(xr[c]) - mu) * rs);
        }
        group_sum(s, red);
        const float c1 = s[0] / (float)cols, c2 = s[1] / (float)cols;
        for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
            const float u = widen(gr[c]) * (w ? widen(w[c]) : 1.0f);
            dx[r * lddx + c] = narrow<T>(rs * (u - c1 - (widen(xr[c]) - mu) * rs * c2));
        }
    }
}

// Partial column sums: workgroup (i, s) takes 256 columns and every row
// r = s, s + S, ...; part[s][0][c] = dw, part[s][1][c] = db.
template <typename T>
__global__ __launch_bounds__(kThreads) void ln_bwd_cols_kernel(const T* __restrict__ dy, int64_t lddy,
                                                               const T* __restrict__ x, int64_t rows, int64_t cols,
                                                               int64_t ldx, const float* __restrict__ mean,
                                                               const float* __restrict__ rstd,
                                                               float* __restrict__ part)
{
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= cols) return;
    float sw = 0.0f, sb = 0.0f;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const float g = widen(dy[r * lddy + c]);
        sw += g * ((widen(x[r * ldx + c]) - mean[r]) * rstd[r]);
        sb += g;
    }
    part[((int64_t)blockIdx.y * 2) * cols + c] = sw;
    part[((int64_t)blockIdx.y * 2 + 1) * cols + c] = sb;
}

template <typename W>
__global__ __launch_bounds__(kThreads) void ln_bwd_join_kernel(const float* __restrict__ part, int64_t parts,
                                                               int64_t cols, W* __restrict__ dw, W* __restrict__ db)
{
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= cols) return;
    float sw = 0.0f, sb = 0.0f;
    for (int64_t s = 0; s < parts; ++s) {
        sw += part[2 * s * cols + c];
        sb += part[(2 * s + 1) * cols + c];
    }
    if (dw) dw[c] = narrow<W>(sw);
    if (db) db[c] = narrow<W>(sb);
}

int64_t row_parts(int64_t rows) { return rows < 256 ? (rows < 1 ? 1 : rows) : 256; }

template <typename T, typename W>
void forward(const void* x, int64_t rows, int64_t cols, int64_t ldx, const void* w, const void* b, float eps, void* y,
             int64_t ldy, float* mean, float* rstd, hipStream_t st)
{
    const dim3 grid((uint32_t)(rows < kMaxRowGroups ? rows : kMaxRowGroups));
    hipLaunchKernelGGL((ln_fwd_kernel<T, W>), grid, dim3(kThreads), 0, st, (const T*)x, rows, cols, ldx, (const W*)w,
                       (const W*)b, eps, (T*)y, ldy, mean, rstd);
}

template <typename T, typename W>
void backward(const void* dy, int64_t lddy, const void* x, int64_t rows, int64_t cols, int64_t ldx, const float* mean,
              const float* rstd, const void* w, void* dx, int64_t lddx, void* dw, void* db, float* ws, hipStream_t st)
{
    const dim3 grid((uint32_t)(rows < kMaxRowGroups ? rows : kMaxRowGroups));
    if (dx && rows > 0)
        hipLaunchKernelGGL((ln_bwd_dx_kernel<T, W>), grid, dim3(kThreads), 0, st, (const T*)dy, lddy, (const T*)x,
                           rows, cols, ldx, mean, rstd, (const W*)w, (T*)dx, lddx);
    if (!dw && !db) return;
    const int64_t parts = row_parts(rows);
    const dim3 cgrid((uint32_t)((cols + kThreads - 1) / kThreads), (uint32_t)parts);
    hipLaunchKernelGGL((ln_bwd_cols_kernel<T>), cgrid, dim3(kThreads), 0, st, (const T*)dy, lddy, (const T*)x, rows,
                       cols, ldx, mean, rstd, ws);
    hipLaunchKernelGGL((ln_bwd_join_kernel<W>), dim3(cgrid.x), dim3(kThreads), 0, st, ws, parts, cols, (W*)dw,
                       (W*)db);
}

}  // namespace

void launch_layer_norm_forward(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const void* w,
                               const void* b, int w_dtype, float eps, void* y, int64_t ldy, float* mean, float* rstd,
                               hipStream_t st)
{
    if (x_dtype == FP8Q_BF16) {
        if (w_dtype == FP8Q_BF16) forward<uint16_t, uint16_t>(x, rows, cols, ldx, w, b, eps, y, ldy, mean, rstd, st);
        else forward<uint16_t, float>(x, rows, cols, ldx, w, b, eps, y, ldy, mean, rstd, st);
    } else {
        if (w_dtype == FP8Q_BF16) forward<float, uint16_t>(x, rows, cols, ldx, w, b, eps, y, ldy, mean, rstd, st);
        else forward<float, float>(x, rows, cols, ldx, w, b, eps, y, ldy, mean, rstd, st);
    }
}

int64_t layer_norm_backward_workspace(int64_t rows, int64_t cols) { return row_parts(rows) * 2 * cols * 4; }

void launch_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int x_dtype, int64_t rows, int64_t cols,
                                int64_t ldx, const float* mean, const float* rstd, const void* w, int w_dtype,
                                void* dx, int64_t lddx, void* dw, void* db, float* ws, hipStream_t st)
{
    if (x_dtype == FP8Q_BF16) {
        if (w_dtype == FP8Q_BF16)
            backward<uint16_t, uint16_t>(dy, lddy, x, rows, cols, ldx, mean, rstd, w, dx, lddx, dw, db, ws, st);
        else
            backward<uint16_t, float>(dy, lddy, x, rows, cols, ldx, mean, rstd, w, dx, lddx, dw, db, ws, st);
    } else {
        if (w_dtype == FP8Q_BF16)
            backward<float, uint16_t>(dy, lddy, x, rows, cols, ldx, mean, rstd, w, dx, lddx, dw, db, ws, st);
        else
            backward<float, float>(dy, lddy, x, rows, cols, ldx, mean, rstd, w, dx, lddx, dw, db, ws, st);
    }
}

}  // namespace fp8q
