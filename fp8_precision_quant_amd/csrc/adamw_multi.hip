// AdamW over many tensors in one launch, for gfx950: moments in E4M3 with one
// fp32 scale per 128 elements, or in fp32.
//
// Per element the step of adam_math.h (the same roundings as the one-tensor
// step); with E4M3 moments the block is decoded first and re-quantized last.
// The moments of all tensors lie in one buffer, each tensor's on a boundary
// of 128 elements.  A workgroup takes one chunk of 32 blocks (4096 elements)
// of one tensor: the plan's table names it, so a launch over tensors of very
// different sizes has equal pieces and no search.  The pointers of parameters
// and gradients travel in the kernel's arguments (up to 192 tensors a
// launch), so a step needs no copy to the device.
#include "adam_math.h"
#include "ops_internal.h"
#include "row_io.h"

namespace fp8q {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;
static_assert(kAdamwChunk == kThreads / 16 * kUnroll, "a chunk is one workgroup's blocks");

struct AdamwArgs {
    const AdamwTensor* tensors;   // of the table
    const AdamwChunk* chunks;     // this launch's first chunk
    int32_t t0;                   // this launch's first tensor
    void* m;
    float* ms;
    void* v;
    float* vs;
    AdamScalars a;
    float* p[kAdamwPerLaunch];
    const void* g[kAdamwPerLaunch];
};
static_assert(sizeof(AdamwArgs) <= 4096, "kernel arguments");

// eight elements at i0 of a vector of n (past n: zero)
template <typename T>
__device__ __forceinline__ void load8e(const T* x, int64_t i0, int64_t n, float v[8])
{
    constexpr int K = kVec<T>;
#pragma unroll
    for (int h = 0; h < 8 / K; ++h) unpack<T>(load_row(x, i0 + h * K, n), v + h * K);
}

__device__ __forceinline__ void store8f(float* x, int64_t i0, int64_t n, const float v[8])
{
    store_row(x, i0, n, pack<float>(v));
    store_row(x, i0 + 4, n, pack<float>(v + 4));
}

// One 16-lane row per block of 128 elements, 8 elements per lane.
template <typename G, bool E4M3>
__global__ __launch_bounds__(kThreads) void adamw_multi_kernel(AdamwArgs args)
{
    const AdamwChunk ch = args.chunks[blockIdx.x];
    const AdamwTensor t = args.tensors[ch.tensor];
    float* const p = args.p[ch.tensor - args.t0];
    const G* const g = (const G*)args.g[ch.tensor - args.t0];
    if (!g) return;
    const int lane16 = threadIdx.x & 15, group = threadIdx.x >> 4;
    float P[kUnroll][8], Gr[kUnroll][8], Mm[kUnroll][8], V[kUnroll][8];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t blk = (int64_t)ch.block + u * (kThreads / 16) + group;
        const int64_t i0 = blk * kTile + lane16 * 8;
        load8e(p, i0, t.n, P[u]);
        load8e(g, i0, t.n, Gr[u]);
        const int64_t e0 = t.block0 * kTile;
        if constexpr (E4M3) {
            const uint8_t* mq = (const uint8_t*)args.m + e0;
            const uint8_t* vq = (const uint8_t*)args.v + e0;
            uint2 mc = {0, 0}, vc = {0, 0};
            float sm = 0.0f, sv = 0.0f;
            if (i0 < t.n) {
                // (a tensor's moments are padded to whole blocks; what lies
                // past n is dropped below)
                mc = *reinterpret_cast<const uint2*>(mq + i0);
                vc = *reinterpret_cast<const uint2*>(vq + i0);
                sm = args.ms[t.block0 + blk];
                sv = args.vs[t.block0 + blk];
            }
            decode8(mc.x, mc.y, Mm[u]);
            decode8(vc.x, vc.y, V[u]);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                Mm[u][k] = i0 + k < t.n ? Mm[u][k] * sm : 0.0f;
                V[u][k] = i0 + k < t.n ? V[u][k] * sv : 0.0f;
            }
        } else {
            load8e((const float*)args.m + e0, i0, t.n, Mm[u]);
            load8e((const float*)args.v + e0, i0, t.n, V[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t blk = (int64_t)ch.block + u * (kThreads / 16) + group;
        const int64_t i0 = blk * kTile + lane16 * 8;
        const int64_t e0 = t.block0 * kTile;
        float mx = 0.0f, vx = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            adam_update(P[u][k], Gr[u][k], Mm[u][k], V[u][k], args.a);
            if constexpr (E4M3) {
                mx = fmaxf(mx, fabsf(Mm[u][k]));
                vx = fmaxf(vx, fabsf(V[u][k]));
            }
        }
        if constexpr (E4M3) {
            const TileScale tm = make_scale(dpp_max16(mx));
            const TileScale tv = make_scale(dpp_max16(vx));
            uint32_t lo, hi, vlo, vhi;
            quant8(Mm[u], tm, lo, hi);
            quant8(V[u], tv, vlo, vhi);
            if (i0 < t.n) {
                uint8_t* mq = (uint8_t*)args.m + e0;
                uint8_t* vq = (uint8_t*)args.v + e0;
                if (i0 + 8 <= t.n) {
                    *reinterpret_cast<uint2*>(mq + i0) = make_uint2(lo, hi);
                    *reinterpret_cast<uint2*>(vq + i0) = make_uint2(vlo, vhi);
                } else {
                    for (int k = 0; i0 + k < t.n; ++k) {
                        mq[i0 + k] = (uint8_t)((k < 4 ? lo : hi) >> (8 * (k & 3)));
                        vq[i0 + k] = (uint8_t)((k < 4 ? vlo : vhi) >> (8 * (k & 3)));
                    }
                }
                if (lane16 == 0) {
                    args.ms[t.block0 + blk] = tm.s;
                    args.vs[t.block0 + blk] = tv.s;
                }
            }
        } else {
            store8f((float*)args.m + e0, i0, t.n, Mm[u]);
            store8f((float*)args.v + e0, i0, t.n, V[u]);
        }
        store8f(p, i0, t.n, P[u]);
    }
}

}  // namespace

void launch_adamw_multi(const void* table, int64_t table_count, int t0, int count, int64_t chunk0, int64_t chunks,
                        float* const* p, const void* const* g, int g_dtype, int kind, void* m, float* ms, void* v,
                        float* vs, const AdamScalars& a, hipStream_t st)
{
    AdamwArgs args;
    args.tensors = reinterpret_cast<const AdamwTensor*>((const char*)table + sizeof(AdamwHeader));
    args.chunks = reinterpret_cast<const AdamwChunk*>(args.tensors + table_count) + chunk0;
    args.t0 = t0;
    args.m = m;
    args.ms = ms;
    args.v = v;
    args.vs = vs;
    args.a = a;
    for (int i = 0; i < kAdamwPerLaunch; ++i) {
        args.p[i] = i < count ? p[t0 + i] : nullptr;
        args.g[i] = i < count ? g[t0 + i] : nullptr;
    }
    const dim3 grid((uint32_t)chunks);
    if (kind == FP8Q_STATE_E4M3) {
        if (g_dtype == FP8Q_BF16)
            hipLaunchKernelGGL((adamw_multi_kernel<uint16_t, true>), grid, dim3(kThreads), 0, st, args);
        else
            hipLaunchKernelGGL((adamw_multi_kernel<float, true>), grid, dim3(kThreads), 0, st, args);
    } else {
        if (g_dtype == FP8Q_BF16)
            hipLaunchKernelGGL((adamw_multi_kernel<uint16_t, false>), grid, dim3(kThreads), 0, st, args);
        else
            hipLaunchKernelGGL((adamw_multi_kernel<float, false>), grid, dim3(kThreads), 0, st, args);
    }
}

}  // namespace fp8q
