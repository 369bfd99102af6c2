// Host-side helpers of the C-ABI layers (api.hip, ops_api.hip): sizes,
// alignment, the device check and the status of a launch.
#pragma once

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "fp8q_internal.h"

namespace fp8q {
namespace host {

constexpr int64_t kTile = 128;   // elements of a scale tile
constexpr int64_t kMaxIndex = (int64_t)1 << 31;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int elem_size(int dtype) { return dtype == FP8Q_BF16 ? 2 : 4; }

inline bool dtype_ok(int d) { return d == FP8Q_F32 || d == FP8Q_BF16; }

// Per-device cache: 0 = unknown, 1 = gfx950, 2 = other / query failed.
inline std::atomic<int> g_arch_state[64];

inline int check_device()
{
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
        (void)hipGetLastError();
        return FP8Q_ERR_DEVICE;
    }
    if (dev >= 64) return FP8Q_ERR_DEVICE;
    int st = g_arch_state[dev].load(std::memory_order_acquire);
    if (st == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
            (void)hipGetLastError();
            st = 2;
        } else {
            st = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        }
        g_arch_state[dev].store(st, std::memory_order_release);
    }
    return st == 1 ? FP8Q_OK : FP8Q_ERR_DEVICE;
}

// The hyperparameters of an AdamW step are in range.
inline bool adam_hyper_ok(double lr, double beta1, double beta2, double eps, double weight_decay, int64_t step)
{
    return beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0 && step >= 1 && std::isfinite(lr) &&
           std::isfinite(eps) && std::isfinite(weight_decay);
}

// The step's derived scalars: computed in double, each rounded once to fp32.
inline AdamScalars adam_scalars(double lr, double beta1, double beta2, double eps, double weight_decay, int64_t step)
{
    AdamScalars a;
    a.b1 = (float)beta1;
    a.b2 = (float)beta2;
    a.omb1 = (float)(1.0 - beta1);
    a.omb2 = (float)(1.0 - beta2);
    a.decay = (float)(1.0 - lr * weight_decay);
    a.step_size = (float)(lr / (1.0 - std::pow(beta1, (double)step)));
    a.bc2_sqrt = (float)std::sqrt(1.0 - std::pow(beta2, (double)step));
    a.eps = (float)eps;
    return a;
}

// A pending launch error; with FP8Q_CHECK=1 the stream is also synchronized
// so that an error of the work itself is reported by the call that enqueued it.
inline int launch_status(hipStream_t stream)
{
    if (hipGetLastError() != hipSuccess) return FP8Q_ERR_LAUNCH;
    if (fp8q::debug_checks_enabled() && hipStreamSynchronize(stream) != hipSuccess) {
        (void)hipGetLastError();
        return FP8Q_ERR_LAUNCH;
    }
    return FP8Q_OK;
}

}  // namespace host
}  // namespace fp8q
