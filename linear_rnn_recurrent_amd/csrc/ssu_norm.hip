// Root-mean-square norm of rows, with the residual's addition before it, a gate
// before or behind it, and an output in a float type or in e4m3 with scales:
//   h = x + residual;  y = h rsqrt(mean h^2 + eps) w;  code = e4m3(y / s), s = max |y| / 448
// Every tensor is read and written once: the span of columns that a sum or a
// maximum runs over (the group, or the block of a scale where that is larger)
// stays in registers between its passes. HBM bounds it, with the vector ALU close
// behind where there is a gate: 4099 rows of 2048 with a residual to e4m3 take 14.7 us (59 MB,
// 4.0 TB/s), 4096 x 32 heads of 128 with a gate 20.3 (101 MB, 5.0 TB/s), 64 rows of 5120 7.3
// a call and 5.7 in a graph (a launch and one chain of loads).
//
// A span belongs to a team of threads, each with NV vectors of eight columns,
// vector m + TEAM j for thread m, so that a load instruction takes consecutive
// memory. Spans of up to 512 columns have teams of 1 to 64 lanes (several spans a
// wave, sums by lane exchange); longer ones have a workgroup, whose waves meet
// once in LDS for each sum. The smaller of group and block is a power of two of at most 64
// vectors, which lie in consecutive lanes of one wave.
#include "ssu_device.h"
#include "ssu_dpp.h"
#include "ssu_internal.h"

namespace ssu {
namespace {

typedef float nm_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 nm_bf16x2 __attribute__((ext_vector_type(2)));

// z / (1 + e^-z) by the hardware's 2^x and reciprocal, an ulp each. The argument of 2^x is rounded
// once: of a gate far below 0, whose e^-z counts, |z| 2^-24 of its value
__device__ __forceinline__ float gate_of(float z)
{
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}

// Eight values of runtime type dt as their bits, converted later so that the
// loads of all tensors are in flight together
struct Raw8 {
    u32x4 w[2];
};

// The same 16 bytes at an element's alignment: global memory takes them in one access
typedef u32x4 Words4 __attribute__((aligned(4)));
typedef u32x4 Halves8 __attribute__((aligned(2)));
typedef u32x2 Bytes8 __attribute__((aligned(1)));

template <bool VEC>
__device__ __forceinline__ Raw8 ld_raw8(const void *p, int64_t i, int dt, int n)
{
    Raw8 r = {};
    if constexpr (VEC) {
        if (dt == kF32) {
            const u32x4 *q = reinterpret_cast<const u32x4 *>(static_cast<const float *>(p) + i);
            r.w[0] = q[0];
            r.w[1] = q[1];
        } else {
            r.w[0] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p) + i);
        }
    } else if (n == 8) {
        if (dt == kF32) {
            const Words4 *q = reinterpret_cast<const Words4 *>(static_cast<const float *>(p) + i);
            r.w[0] = q[0];
            r.w[1] = q[1];
        } else {
            r.w[0] = *reinterpret_cast<const Halves8 *>(static_cast<const uint16_t *>(p) + i);
        }
    } else if (dt == kF32) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n)
                r.w[e / 4][e % 4] = static_cast<const uint32_t *>(p)[i + e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n)
                r.w[0][e / 2] |= (uint32_t)static_cast<const uint16_t *>(p)[i + e] << (16 * (e % 2));
    }
    return r;
}

__device__ __forceinline__ void cvt_raw8(const Raw8 &r, int dt, float (&v)[8])
{
    if (dt == kF32) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = __uint_as_float(r.w[e / 4][e % 4]);
    } else if (dt == kBF16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(r.w[0][e] << 16);
            v[2 * e + 1] = __uint_as_float(r.w[0][e] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = f16_to_f32(r.w[0][e] & 0xffffu);
            v[2 * e + 1] = f16_to_f32(r.w[0][e] >> 16);
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void st_vec8(void *p, int64_t i, int dt, const float (&v)[8], int n)
{
    if (VEC || n == 8) {
        if (dt == kF32) {
            float *q = static_cast<float *>(p) + i;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const u32x4 w = {__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]),
                                 __float_as_uint(v[4 * k + 2]), __float_as_uint(v[4 * k + 3])};
                if constexpr (VEC)
                    reinterpret_cast<u32x4 *>(q)[k] = w;
                else
                    reinterpret_cast<Words4 *>(q)[k] = w;
            }
        } else {
            u32x4 w;
            if (dt == kBF16) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(
                                                            (nm_f32x2){v[2 * k], v[2 * k + 1]}, nm_bf16x2));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = f32_to_f16(v[2 * k]) | (f32_to_f16(v[2 * k + 1]) << 16);
            }
            uint16_t *q = static_cast<uint16_t *>(p) + i;
            if constexpr (VEC)
                *reinterpret_cast<u32x4 *>(q) = w;
            else
                *reinterpret_cast<Halves8 *>(q) = w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n)
                st_io(p, i + e, v[e], dt);
    }
}

// v / scale, given 1 / scale: a product and its remainder's, as a division rounds
__device__ __forceinline__ float over(float v, float scale, float inv)
{
    const float q = v * inv;
    const float fix = fmaf(fmaf(-q, scale, v), inv, q);
    return fix == fix ? fix : q;  // infinite v or scale: their quotient as it came
}

template <bool VEC>
__device__ __forceinline__ void st_e4m3(void *p, int64_t i, const float (&v)[8], float scale, float inv,
                                        int n)
{
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int c = __builtin_amdgcn_cvt_pk_fp8_f32(over(v[4 * k], scale, inv),
                                                      over(v[4 * k + 1], scale, inv), 0, false);
        w[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(over(v[4 * k + 2], scale, inv),
                                                         over(v[4 * k + 3], scale, inv), c, true);
    }
    uint8_t *q = static_cast<uint8_t *>(p) + i;
    if constexpr (VEC) {
        *reinterpret_cast<u32x2 *>(q) = u32x2{w[0], w[1]};
    } else if (n == 8) {
        *reinterpret_cast<Bytes8 *>(q) = u32x2{w[0], w[1]};
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n)
                q[e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
    }
}

// Sum, and maximum of bits, over aligned runs of `width` lanes (a power of two);
// as unsigned numbers the bits of magnitudes order as they do, NaN above all.
__device__ __forceinline__ float lanes_sum(float v, int width)
{
    if (width == 64)
        return wave_sum(v);
    for (int m = 1; m < width; m <<= 1)
        v += __shfl_xor(v, m, 64);
    return v;
}
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int width)
{
    for (int m = 1; m < width; m <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, m, 64);
        v = o > v ? o : v;
    }
    return v;
}

// WG: the span belongs to the workgroup, otherwise to `team` lanes. vecs: vectors of a span.
template <int NV, bool WG, bool VEC>
__global__ __launch_bounds__(1024) void norm_kernel(NormParams p, int span, int per_row, int team,
                                                    int vecs, int sub, int64_t spans)
{
    __shared__ float part_f[16];
    __shared__ uint32_t part_u[16];
    constexpr bool EARLY = NV <= 2;  // z and the weights loaded with the rest (registers for four vectors do not reach)
    const int nt = blockDim.x;
    const int m = WG ? threadIdx.x : (threadIdx.x & (team - 1));
    // fewer than 2^32 threads: 32 bits
    const uint32_t s = WG ? blockIdx.x : (blockIdx.x * (uint32_t)nt + threadIdx.x) >> __builtin_ctz(team);
    // lanes past the last span keep their wave whole for the exchanges
    const bool live = s < spans;
    const uint32_t row = !live ? 0 : per_row == 1 ? s : s / (uint32_t)per_row;
    const uint32_t b32 = p.tokens == p.rows ? 0 : row / (uint32_t)p.tokens;
    const int64_t b = b32, t = row - b32 * (uint32_t)p.tokens;
    const int c0 = live ? (int)(s - row * (uint32_t)per_row) * span : 0;
    const float inv_group = 1.0f / (float)p.group;
    // of the weights: a span begins a group, and smaller groups are powers of two
    auto weight_at = [&](int c) {
        return p.weight_columns == p.columns ? c : p.group >= span ? c - c0 : (c - c0) & (p.group - 1);
    };

    Raw8 rx[NV], rr[NV], rz[NV], rw[NV];
    int cols[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = m + (WG ? nt : team) * j;
        cols[j] = !live || i >= vecs ? 0 : VEC ? 8 : min(8, span - 8 * i);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (cols[j] > 0) {
            const int c = c0 + 8 * (m + (WG ? nt : team) * j);
            rx[j] = ld_raw8<VEC>(p.x, b * p.x_bs + t * p.x_ts + c, p.io_dtype, cols[j]);
            if (p.residual)
                rr[j] = ld_raw8<VEC>(p.residual, b * p.r_bs + t * p.r_ts + c, p.residual_dtype, cols[j]);
            if (EARLY && p.z)
                rz[j] = ld_raw8<VEC>(p.z, b * p.z_bs + t * p.z_ts + c, p.io_dtype, cols[j]);
            if (EARLY)
                rw[j] = ld_raw8<VEC>(p.weight, weight_at(c),
                                     p.weight_dtype, cols[j]);
        }
    }

    float h[NV][8];
    float sq[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        sq[j] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            h[j][e] = 0.0f;
        if (cols[j] > 0) {
            const int c = c0 + 8 * (m + (WG ? nt : team) * j);
            cvt_raw8(rx[j], p.io_dtype, h[j]);
            if (p.residual) {
                float r[8];
                cvt_raw8(rr[j], p.residual_dtype, r);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    h[j][e] += r[e];
                st_vec8<VEC>(p.residual, b * p.r_bs + t * p.r_ts + c, p.residual_dtype, h[j], cols[j]);
            }
            if (p.z && p.gate_first) {
                float z[8];
                if (!EARLY)
                    rz[j] = ld_raw8<VEC>(p.z, b * p.z_bs + t * p.z_ts + c, p.io_dtype, cols[j]);
                cvt_raw8(rz[j], p.io_dtype, z);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    h[j][e] *= gate_of(z[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sq[j] += VEC || e < cols[j] ? h[j][e] * h[j][e] : 0.0f;
        }
    }

    // sums of squares of the groups
    if (p.group < span) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            sq[j] = lanes_sum(sq[j], sub);
    } else {
        float a = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            a += sq[j];
        if constexpr (WG) {
            a = wave_sum(a);
            if (nt > 64) {
                if ((threadIdx.x & 63) == 0)
                    part_f[threadIdx.x >> 6] = a;
                __syncthreads();
                a = 0.0f;
                for (int w = 0; w < nt / 64; ++w)
                    a += part_f[w];
            }
        } else {
            a = lanes_sum(a, team);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
            sq[j] = a;
    }

    const float one = p.unit_offset ? 1.0f : 0.0f;
    // A block within one group: its codes are those of h w over their maximum, without the
    // root, and so without two of the four roundings before the code (264 codes of 10^8 differ
    // from the formula's, 326 with them)
    const bool apart = p.out_dtype == kE4m3 && p.block <= p.group;
    uint32_t most[NV];
    float root[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        most[j] = 0;
        // a Newton step behind the hardware's root: codes flip where y is off by an ulp or two
        const float mean = sq[j] * inv_group + p.eps;
        float inv = __builtin_amdgcn_rsqf(mean);
        const float half = 0.5f * inv;
        inv = mean > 0x1p-100f && mean < 0x1p100f ? fmaf(half, fmaf(-mean * inv, inv, 1.0f), inv) : inv;
        root[j] = apart ? inv : 1.0f;
        if (apart)
            inv = 1.0f;
        if (cols[j] > 0) {
            float w[8], z[8];
            if (!EARLY) {
                const int c = c0 + 8 * (m + (WG ? nt : team) * j);
                rw[j] = ld_raw8<VEC>(p.weight, weight_at(c),
                                     p.weight_dtype, cols[j]);
                if (p.z && !p.gate_first)
                    rz[j] = ld_raw8<VEC>(p.z, b * p.z_bs + t * p.z_ts + c, p.io_dtype, cols[j]);
            }
            cvt_raw8(rw[j], p.weight_dtype, w);
            if (p.z && !p.gate_first)
                cvt_raw8(rz[j], p.io_dtype, z);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float y = h[j][e] * inv * (one + w[e]);
                if (p.z && !p.gate_first)
                    y *= gate_of(z[e]);
                h[j][e] = y;
            }
            if (p.out_dtype == kE4m3) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t mag = VEC || e < cols[j] ? __float_as_uint(h[j][e]) & 0x7fffffffu : 0u;
                    most[j] = mag > most[j] ? mag : most[j];
                }
            }
        }
    }
    if (p.out_dtype != kE4m3) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (cols[j] > 0)
                st_vec8<VEC>(p.out, b * p.out_bs + t * p.out_ts + c0 + 8 * (m + (WG ? nt : team) * j),
                             p.out_dtype, h[j], cols[j]);
        return;
    }

    // maxima of the scales' blocks
    if (p.block < span) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            most[j] = lanes_max(most[j], sub);
    } else {
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            a = most[j] > a ? most[j] : a;
        a = lanes_max(a, WG ? 64 : team);
        if constexpr (WG) {
            if (nt > 64) {
                if ((threadIdx.x & 63) == 0)
                    part_u[threadIdx.x >> 6] = a;
                __syncthreads();
                for (int w = 0; w < nt / 64; ++w)
                    a = part_u[w] > a ? part_u[w] : a;
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
            most[j] = a;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (cols[j] > 0) {
            const int i = m + (WG ? nt : team) * j, c = c0 + 8 * i;
            const float top = __uint_as_float(most[j]);
            const float a = top * root[j] / 448.0f;
            const float scale = a < 0x1p-126f ? 0x1p-126f : a;  // a NaN stays
            const bool fine = top > 0x1p-100f && top < 0x1p100f && a >= 0x1p-126f;
            const float by = fine ? top / 448.0f : scale, times = fine ? 1.0f : root[j];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[j][e] *= times;
            st_e4m3<VEC>(p.out, b * p.out_bs + t * p.out_ts + c, h[j], by, 1.0f / by, cols[j]);
            const int in = p.block >= span ? 8 * i : (8 * i) & (p.block - 1);
            if (in == 0)
                p.scales[(int64_t)row * (p.columns / p.block) + c / p.block] = scale;
        }
}

bool norm_aligned(const NormParams &p, int span)
{
    auto fine = [](const void *t, int64_t bs, int64_t ts, int dt) {
        const int64_t e = dt == kF32 ? 4 : dt == kE4m3 ? 1 : 2, to = e == 1 ? 8 : 16;
        return !t || ((uintptr_t)t | (uintptr_t)(bs * e) | (uintptr_t)(ts * e)) % to == 0;
    };
    return span % 8 == 0 && p.group % 8 == 0 && fine(p.x, p.x_bs, p.x_ts, p.io_dtype) &&
           fine(p.z, p.z_bs, p.z_ts, p.io_dtype) &&
           fine(p.residual, p.r_bs, p.r_ts, p.residual_dtype) &&
           fine(p.out, p.out_bs, p.out_ts, p.out_dtype) && fine(p.weight, 0, 0, p.weight_dtype);
}

template <int NV, bool WG>
hipError_t launch_norm_nv(const NormParams &p, int span, int team, int threads, hipStream_t stream)
{
    const int64_t spans = p.rows * (p.columns / span);
    const int vecs = (span + 7) / 8, per_row = p.columns / span;
    const int sub = (p.out_dtype == kE4m3 ? min(p.group, p.block) : p.group) / 8;
    const __int128 groups = WG ? spans : ((__int128)spans * team + threads - 1) / threads;
    if (!launchable(groups, threads))
        return hipErrorInvalidConfiguration;
    if (norm_aligned(p, span))
        norm_kernel<NV, WG, true><<<dim3((uint32_t)groups), threads, 0, stream>>>(p, span, per_row, team, vecs,
                                                                                  sub, spans);
    else
        norm_kernel<NV, WG, false><<<dim3((uint32_t)groups), threads, 0, stream>>>(p, span, per_row, team, vecs,
                                                                                   sub, spans);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormParams &given, hipStream_t stream)
{
    (void)hipGetLastError();  // report only this launch's status
    NormParams p = given;
    if (p.rows > 0x7fffffff)
        return hipErrorInvalidConfiguration;
    const int64_t n = p.tokens;
    if (n == 1 || p.rows == n ||
        (p.x_bs == n * p.x_ts && p.out_bs == n * p.out_ts && (!p.z || p.z_bs == n * p.z_ts) &&
         (!p.residual || p.r_bs == n * p.r_ts))) {  // one row after the other: no batch
        if (n == 1) {
            p.x_ts = p.x_bs;
            p.z_ts = p.z_bs;
            p.r_ts = p.r_bs;
            p.out_ts = p.out_bs;
        }
        p.tokens = (int32_t)p.rows;
    }
    const int span = p.out_dtype == kE4m3 && p.block > p.group ? p.block : p.group;
    const int vecs = (span + 7) / 8;
    if (vecs <= 64) {
        int team = 1;
        while (team < vecs)
            team *= 2;
        return launch_norm_nv<1, false>(p, span, team, 256, stream);
    }
    // two vectors a thread, four where a workgroup's 1,024 threads do not reach
    const int nv = vecs <= 2048 ? 2 : 4;
    const int threads = ((vecs + nv - 1) / nv + 63) / 64 * 64;
    return nv == 2 ? launch_norm_nv<2, true>(p, span, 0, threads, stream)
                   : launch_norm_nv<4, true>(p, span, 0, threads, stream);
}

}  // namespace ssu
