// What the scan's kernels share: small device helpers, and the plan of a call
// (ssu_scan_plan.h).
#pragma once

#include <atomic>
#include <type_traits>
#include <utility>

#include "ssu_device.h"
#include "ssu_dpp.h"
#include "ssu_internal.h"
#include "ssu_scan_plan.h"

namespace ssu {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Rounds to nearest even in one instruction (bf16: v_cvt_pk_bf16_f32).
template <typename T>
__device__ __forceinline__ void put(void *at, float v)
{
    if constexpr (sizeof(T) == 4)
        *static_cast<float *>(at) = v;
    else if constexpr (__is_same(T, bf16_t))
        *static_cast<__bf16 *>(at) = (__bf16)v;
    else
        *static_cast<_Float16 *>(at) = (_Float16)v;
}

// v sigmoid(v) on the hardware exp2 and reciprocal (1 ulp each).
__device__ __forceinline__ float silu_hw(float v)
{
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// A's entry for exp2; an infinite one as the largest finite, which decays as fast
// and leaves the state where dt' is 0 (tokens behind a row's end).
__device__ __forceinline__ float log2_rate(float a)
{
    const float r = a * kLog2e;
    return __builtin_isinf(r) ? copysignf(3.402823466e38f, r) : r;
}

// The decay over several tokens whose dt' sum to `sum`. Growth past the range of
// fp32 (A dt' > 0) is its largest value: the tokens one by one leave a 0 at 0. (A NaN
// is in the tokens' own end as well.)
__device__ __forceinline__ float whole_decay(float rate, float sum)
{
    return fminf(__builtin_amdgcn_exp2f(rate * sum), 3.402823466e38f);
}

__device__ __forceinline__ int row_tokens(const ScanParams &p, int b, int *row)
{
    *row = p.idx ? p.idx[b] : b;
    return *row < 0 ? 0 : (p.ctx ? clamp_len(p.ctx[b], p.seq_len) : p.seq_len);
}

// An element, or four, of a tensor by the size of its elements, as raw bits;
// which 16-bit type it is is a (uniform) choice made after the load, so that
// all loads of a token are issued before any is waited for. SZ 0: the size is a
// choice as well, and the four need no alignment.
template <int SZ>
__device__ __forceinline__ uint32_t raw1(const void *p, int64_t i, int dt)
{
    if (SZ == 4 || (SZ == 0 && dt == kF32))
        return static_cast<const uint32_t *>(p)[i];
    return static_cast<const uint16_t *>(p)[i];
}
template <int SZ>
__device__ __forceinline__ float cvt1(uint32_t w, int dt)
{
    if (SZ == 4 || (SZ == 0 && dt == kF32))
        return __uint_as_float(w);
    const float bf = __uint_as_float(w << 16), hf = f16_to_f32(w & 0xffffu);
    return dt == kBF16 ? bf : hf;
}
struct Raw4x {
    uint32_t w[4];
};
template <int SZ>
__device__ __forceinline__ Raw4x raw4(const void *p, int64_t i, int dt)
{
    Raw4x r;
    if constexpr (SZ == 4) {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(static_cast<const uint32_t *>(p) + i);
        r.w[0] = v[0], r.w[1] = v[1], r.w[2] = v[2], r.w[3] = v[3];
    } else if constexpr (SZ == 2) {
        const u32x2 v = *reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(p) + i);
        r.w[0] = v[0], r.w[1] = v[1], r.w[2] = 0, r.w[3] = 0;  // split by cvt4
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r.w[j] = raw1<0>(p, i + j, dt);
    }
    return r;
}
template <int SZ>
__device__ __forceinline__ void cvt4(const Raw4x &r, int dt, float (&v)[4])
{
    if constexpr (SZ == 2) {
        v[0] = cvt1<2>(r.w[0], dt), v[1] = cvt1<2>(r.w[0] >> 16, dt);
        v[2] = cvt1<2>(r.w[1], dt), v[3] = cvt1<2>(r.w[1] >> 16, dt);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = cvt1<SZ>(r.w[j], dt);
    }
}
// Four adjacent state entries, aligned to four, as floats.
__device__ __forceinline__ void ld_state4(const ScanParams &p, int64_t i, float (&v)[4])
{
    if (p.state_dtype == kF32)
        cvt4<4>(raw4<4>(p.state, i, kF32), kF32, v);
    else
        cvt4<2>(raw4<2>(p.state, i, p.state_dtype), p.state_dtype, v);
}
template <int SZ>
__device__ __forceinline__ void st1(void *p, int64_t i, float v, int dt)
{
    if (SZ == 4 || (SZ == 0 && dt == kF32)) {
        static_cast<float *>(p)[i] = v;
        return;
    }
    const uint16_t bf = __builtin_bit_cast(uint16_t, (__bf16)v);
    const uint16_t hf = __builtin_bit_cast(uint16_t, (_Float16)v);
    static_cast<uint16_t *>(p)[i] = dt == kBF16 ? bf : hf;
}

}  // namespace

}  // namespace ssu
