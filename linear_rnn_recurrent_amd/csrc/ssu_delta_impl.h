// What the evaluations of the gated delta rule share.
#pragma once

#include "ssu_device.h"
#include "ssu_dpp.h"
#include "ssu_internal.h"

namespace ssu {
namespace {

constexpr float kDeltaEps = 1e-6f;  // of the norms of q and k

struct DeltaGate {
    float alpha, beta;
};

// The logarithm of a token's decay
__device__ __forceinline__ float delta_log_decay(const DeltaParams &p, float A, float bias, float a)
{
    return p.A_log ? A * softplus_f32(a + bias) : a;
}

__device__ __forceinline__ float delta_beta(const DeltaParams &p, float b)
{
    return p.A_log ? 1.0f / (1.0f + expf(-b)) : b;
}

// A: -exp(A_log[h]), bias: dt_bias[h] (both unused without A_log)
__device__ __forceinline__ DeltaGate delta_gate(const DeltaParams &p, float A, float bias, float a,
                                                float b)
{
    return {expf(delta_log_decay(p, A, bias, a)), delta_beta(p, b)};
}

// Four state entries, aligned, past the caches (a pool is far larger than them)
__device__ __forceinline__ void delta_st_state(float *s, const float (&t)[4])
{
    __builtin_nontemporal_store(u32x4{__float_as_uint(t[0]), __float_as_uint(t[1]),
                                      __float_as_uint(t[2]), __float_as_uint(t[3])},
                                reinterpret_cast<u32x4 *>(s));
}
__device__ __forceinline__ void delta_st_state(_Float16 *s, const float (&t)[4])
{
    __builtin_nontemporal_store(u32x2{f32_to_f16(t[0]) | (f32_to_f16(t[1]) << 16),
                                      f32_to_f16(t[2]) | (f32_to_f16(t[3]) << 16)},
                                reinterpret_cast<u32x2 *>(s));
}
__device__ __forceinline__ void delta_st_state(bf16_t *s, const float (&t)[4])
{
    __builtin_nontemporal_store(u32x2{f32_to_bf16(t[0]) | (f32_to_bf16(t[1]) << 16),
                                      f32_to_bf16(t[2]) | (f32_to_bf16(t[3]) << 16)},
                                reinterpret_cast<u32x2 *>(s));
}

// Whether every token's rows of q, k, v and out start at a multiple of `bytes`
inline bool delta_rows_aligned(const DeltaParams &p, int bytes)
{
    const int64_t e = p.io_dtype == kF32 ? 4 : 2;
    auto fine = [&](const void *t, int64_t bs, int64_t ts) {
        return ((uintptr_t)t | (uintptr_t)(bs * e) | (uintptr_t)(ts * e)) % bytes == 0;
    };
    return fine(p.k, p.k_bs, p.k_ts) && fine(p.v, p.v_bs, p.v_ts) &&
           (!p.out || (fine(p.q, p.q_bs, p.q_ts) && fine(p.out, p.out_bs, p.out_ts)));
}

}  // namespace
}  // namespace ssu
