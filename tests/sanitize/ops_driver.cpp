// Calls the entry points of include/fp8q_ops.h with arguments that their
// host-side validation must refuse, and fills and checks AdamW tables in
// exactly sized buffers.  Built with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code (device code not compiled).
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../include/fp8q_ops.h"

namespace {

int failures = 0;

void expect(int64_t got, int64_t want, const char* what)
{
    if (got != want) {
        std::fprintf(stderr, "%s: got %lld, want %lld\n", what, (long long)got, (long long)want);
        ++failures;
    }
}

uint8_t* const P = reinterpret_cast<uint8_t*>(uintptr_t(1) << 20);   // never dereferenced
uint8_t* const U = P + 1;
float* const F = reinterpret_cast<float*>(P);
float* const FU = reinterpret_cast<float*>(U);
int8_t* const Q = reinterpret_cast<int8_t*>(P);
constexpr int64_t kHuge = INT64_MAX;

}  // namespace

int main()
{
    // layer norm
    expect(fp8q_layer_norm_forward(P, 7, 4, 8, 8, P, P, 0, 1e-5, P, 8, F, F, nullptr), FP8Q_ERR_UNSUPPORTED, "lnf dtype");
    expect(fp8q_layer_norm_forward(P, 0, kHuge, kHuge, kHuge, P, P, 0, 1e-5, P, kHuge, F, F, nullptr), FP8Q_ERR_SHAPE,
           "lnf huge");
    expect(fp8q_layer_norm_forward(P, 0, 4, 8, 8, P, P, 0, NAN, P, 8, F, F, nullptr), FP8Q_ERR_UNSUPPORTED, "lnf eps");
    expect(fp8q_layer_norm_forward(P, 0, 4, 8, 8, P, P, 0, 0.0, U, 8, F, F, nullptr), FP8Q_ERR_ALIGN, "lnf align");
    expect(fp8q_layer_norm_backward_workspace(INT64_MIN, 4), 0, "lnb workspace rows");
    expect(fp8q_layer_norm_backward_workspace(4, kHuge), 0, "lnb workspace cols");
    expect(fp8q_layer_norm_backward(P, 8, P, 1, 4, 8, 8, F, F, P, 1, P, 8, P, P, P, 1, nullptr), FP8Q_ERR_SHAPE,
           "lnb workspace size");
    expect(fp8q_layer_norm_backward(P, 8, P, 1, kHuge, 8, 8, F, F, P, 1, P, 8, P, P, P, kHuge, nullptr), FP8Q_ERR_SHAPE,
           "lnb rows");
    expect(fp8q_layer_norm_backward(P, 8, P, 1, 4, 8, 8, FU, F, P, 1, P, 8, P, P, P, kHuge, nullptr), FP8Q_ERR_ALIGN,
           "lnb align");

    // AdamW tables: exact buffers, so a write past the end is seen
    for (int64_t count : {0, 1, 2, 57, 300}) {
        std::vector<int64_t> n(count);
        for (int64_t i = 0; i < count; ++i) n[i] = (i * 7919) % 20000;
        const int64_t bytes = fp8q_adamw_table_bytes(count, n.data());
        std::vector<int64_t> table(bytes / 8);
        expect(fp8q_adamw_table_fill(count, n.data(), table.data(), bytes), FP8Q_OK, "table fill");
        expect(fp8q_adamw_table_fill(count, n.data(), table.data(), bytes - 8), FP8Q_ERR_SHAPE, "table size");
        std::vector<float*> p(count, F);
        std::vector<const void*> g(count, F);
        expect(fp8q_adamw_multi_step(table.data(), P, p.data(), g.data(), 3, FP8Q_STATE_F32, P, F, P, F, 1e-3, 0.9, 0.999,
                                     1e-8, 0.0, 1, nullptr), FP8Q_ERR_UNSUPPORTED, "adamw dtype");
        if (count < 2) continue;
        p[count - 1] = FU;
        expect(fp8q_adamw_multi_step(table.data(), P, p.data(), g.data(), FP8Q_F32, FP8Q_STATE_F32, P, F, P, F, 1e-3, 0.9,
                                     0.999, 1e-8, 0.0, 1, nullptr), FP8Q_ERR_ALIGN, "adamw parameter");
        p[count - 1] = nullptr;
        expect(fp8q_adamw_multi_step(table.data(), P, p.data(), g.data(), FP8Q_F32, FP8Q_STATE_E4M3, P, F, P, F, 1e-3, 0.9,
                                     0.999, 1e-8, 0.0, 1, nullptr), FP8Q_ERR_NULL, "adamw null parameter");
    }
    const int64_t bad[3] = {kHuge, kHuge, kHuge};
    expect(fp8q_adamw_table_bytes(3, bad), -1, "table huge sizes");
    expect(fp8q_adamw_table_bytes(kHuge, bad), -1, "table huge count");

    // int8
    expect(fp8q_int8_quant_rows(P, 0, 4, kHuge, kHuge, Q, kHuge, F, nullptr), FP8Q_ERR_SHAPE, "quant cols");
    expect(fp8q_int8_quant_rows(P, 0, 4, 100, 100, Q, 104, F, nullptr), FP8Q_ERR_ALIGN, "quant ldq");
    expect(fp8q_int8_gemm_workspace(kHuge, kHuge, kHuge), 0, "gemm workspace");
    expect(fp8q_int8_gemm(kHuge, 8, 8, Q, 16, F, Q, 16, F, F, P, 8, 0, nullptr, 0, nullptr), FP8Q_ERR_SHAPE, "gemm M");
    expect(fp8q_int8_gemm(INT32_MAX, INT32_MAX, 8, Q, 16, F, Q, 16, F, F, P, int64_t(1) << 31, 0, nullptr, 0, nullptr),
           FP8Q_ERR_UNSUPPORTED, "gemm tiles");
    expect(fp8q_int8_gemm(4, 8, 8, Q, 16, F, Q, 16, F, F, P, kHuge, 0, nullptr, 0, nullptr), FP8Q_ERR_SHAPE, "gemm ldc");
    expect(fp8q_int8_gemm(4, 8, kHuge, Q, kHuge, F, Q, kHuge, F, F, P, 8, 0, nullptr, 0, nullptr), FP8Q_ERR_UNSUPPORTED,
           "gemm K");
    expect(fp8q_int8_gemm(4, 8, 8, Q, kHuge, F, Q, 16, F, F, P, 8, 0, nullptr, 0, nullptr), FP8Q_ERR_UNSUPPORTED,
           "gemm lda");
    expect(fp8q_int8_gemm(96, 8, 8, Q, 16, F, Q, 16, F, F, P, 8, 0, nullptr, 0, nullptr), FP8Q_ERR_NULL, "gemm ws");
    expect(fp8q_int8_gemm(96, 8, 8, Q, 16, F, Q, 16, F, F, P, 8, 0, P, 4095, nullptr), FP8Q_ERR_SHAPE, "gemm ws size");
    expect(fp8q_int8_gemm(4, 8, 8, Q, 16, F, Q, 16, F, FU, P, 8, 0, nullptr, 0, nullptr), FP8Q_ERR_ALIGN, "gemm bias");

    if (failures) {
        std::fprintf(stderr, "%d case(s) failed\n", failures);
        return 1;
    }
    std::printf("ops driver: all validation cases passed\n");
    return 0;
}
