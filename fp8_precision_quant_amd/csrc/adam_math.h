// The AdamW step's arithmetic, shared by the one-tensor kernel (adam.hip) and
// the many-tensor kernels (adamw_multi.hip).
#pragma once

#include "fp8q_device.h"
#include "fp8q_internal.h"

namespace fp8q {

typedef float v2f __attribute__((ext_vector_type(2)));

// eight E4M3 codes (little-endian in lo, hi) -> fp32 values (exact)
__device__ __forceinline__ void decode8(uint32_t lo, uint32_t hi, float v[8])
{
    const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)lo, false);
    const v2f b = __builtin_amdgcn_cvt_pk_f32_fp8((int)lo, true);
    const v2f c = __builtin_amdgcn_cvt_pk_f32_fp8((int)hi, false);
    const v2f d = __builtin_amdgcn_cvt_pk_f32_fp8((int)hi, true);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
}

// One element of the step: every fp32 operation rounded once, in this order
// (no contraction into FMAs); p, m and v are updated in place.
__device__ __forceinline__ void adam_update(float& p, float g, float& m, float& v, const AdamScalars& a)
{
#pragma clang fp contract(off)
    const float pi = p * a.decay;
    const float t0 = a.b1 * m;
    const float t1 = a.omb1 * g;
    const float mi = t0 + t1;
    const float t2 = a.b2 * v;
    const float t3 = a.omb2 * g;
    const float t4 = t3 * g;
    const float vi = t2 + t4;
    const float r = __builtin_sqrtf(vi);
    const float q = r / a.bc2_sqrt;
    const float den = q + a.eps;
    const float upd = mi / den;
    const float w = a.step_size * upd;
    p = pi - w;
    m = mi;
    v = vi;
}

}  // namespace fp8q
