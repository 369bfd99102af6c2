// Launchers of the operators around the linear layers (layer norm, AdamW over
// many tensors, int8 quantizer and product).  Arguments were validated by the
// C-ABI layer (ops_api.hip); a launcher only enqueues kernels on `st`.
#pragma once

#include "../../include/fp8q_ops.h"
#include "fp8q_internal.h"

namespace fp8q {

void launch_layer_norm_forward(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const void* w,
                               const void* b, int w_dtype, float eps, void* y, int64_t ldy, float* mean, float* rstd,
                               hipStream_t st);

// bytes of scratch that the backward pass's column sums need
int64_t layer_norm_backward_workspace(int64_t rows, int64_t cols);
void launch_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int x_dtype, int64_t rows, int64_t cols,
                                int64_t ldx, const float* mean, const float* rstd, const void* w, int w_dtype,
                                void* dx, int64_t lddx, void* dw, void* db, float* ws, hipStream_t st);

// The table of an AdamW plan: this header, one AdamwTensor per tensor, one
// AdamwChunk per kAdamwChunk scale tiles of each tensor (a workgroup's work).
struct AdamwHeader {
    uint64_t magic;
    int64_t count, chunks, bytes;
};
struct AdamwTensor {
    int64_t n;        // elements
    int64_t block0;   // its first 128-element block in the moments
    int64_t chunk0;   // its first chunk
    int64_t reserved;
};
struct AdamwChunk {
    int32_t tensor;
    uint32_t block;   // first block of the chunk within its tensor
};
constexpr int kAdamwChunk = 32;          // blocks of 128 per chunk
constexpr uint64_t kAdamwMagic = 0x46513841444d5731ull;
constexpr int kAdamwPerLaunch = 192;     // tensors whose pointers travel in one launch's arguments

// tensors [t0, t0 + count), chunks [chunk0, chunk0 + chunks) of the table
void launch_adamw_multi(const void* table, int64_t table_count, int t0, int count, int64_t chunk0, int64_t chunks,
                        float* const* p, const void* const* g, int g_dtype, int kind, void* m, float* ms, void* v,
                        float* vs, const AdamScalars& a, hipStream_t st);

void launch_int8_quant_rows(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, int8_t* q,
                            int64_t ldq, float* s, hipStream_t st);

// bytes of scratch of the product (0: none needed)
int64_t int8_gemm_workspace(int64_t M, int64_t N, int64_t K);
void launch_int8_gemm(int64_t M, int64_t N, int64_t K, const int8_t* a, int64_t lda, const float* sa, const int8_t* b,
                      int64_t ldb, const float* sb, const float* bias, void* c, int64_t ldc, int c_dtype, int32_t* ws,
                      hipStream_t st);

}  // namespace fp8q
