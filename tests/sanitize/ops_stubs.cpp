// Stand-ins for the launchers of the operators (ops_internal.h), linked with
// the host code of their C-ABI layer (ops_api.hip) for the sanitizer run:
// every call of the driver must be refused by validation, so reaching a
// launcher is a failure.  The two scratch sizes are asked during validation
// and answer like the library's (any positive size serves the driver).
#include <cstdio>
#include <cstdlib>

#include "../../fp8_precision_quant_amd/csrc/ops_internal.h"

namespace {
[[noreturn]] void reached(const char* what)
{
    std::fprintf(stderr, "validation let a call through to %s\n", what);
    std::abort();
}
}  // namespace

namespace fp8q {

bool debug_checks_enabled() { return false; }
int64_t layer_norm_backward_workspace(int64_t, int64_t cols) { return 8 * (cols < 1 ? 1 : cols); }
int64_t int8_gemm_workspace(int64_t M, int64_t, int64_t) { return M == 96 ? 4096 : 0; }
void launch_layer_norm_forward(const void*, int, int64_t, int64_t, int64_t, const void*, const void*, int, float, void*,
                               int64_t, float*, float*, hipStream_t)
{
    reached("launch_layer_norm_forward");
}
void launch_layer_norm_backward(const void*, int64_t, const void*, int, int64_t, int64_t, int64_t, const float*,
                                const float*, const void*, int, void*, int64_t, void*, void*, float*, hipStream_t)
{
    reached("launch_layer_norm_backward");
}
void launch_adamw_multi(const void*, int64_t, int, int, int64_t, int64_t, float* const*, const void* const*, int, int,
                        void*, float*, void*, float*, const AdamScalars&, hipStream_t)
{
    reached("launch_adamw_multi");
}
void launch_int8_quant_rows(const void*, int, int64_t, int64_t, int64_t, int8_t*, int64_t, float*, hipStream_t)
{
    reached("launch_int8_quant_rows");
}
void launch_int8_gemm(int64_t, int64_t, int64_t, const int8_t*, int64_t, const float*, const int8_t*, int64_t,
                      const float*, const float*, void*, int64_t, int, int32_t*, hipStream_t)
{
    reached("launch_int8_gemm");
}

}  // namespace fp8q
