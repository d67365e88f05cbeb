// Per-channel selective scan of single tokens and short windows: the kernels of
// ssu_scan.hip's first evaluation, which that file describes.
#include "ssu_scan_impl.h"

namespace ssu {
namespace {

// ---------------------------------------------------------------------------
// Rows: LPC lanes per channel
// ---------------------------------------------------------------------------
// Four state entries (aligned to four elements), past the caches: each is read
// and written once a call.
template <typename ST>
__device__ __forceinline__ typename Raw4<ST>::type ld_state4(const ST *p)
{
    return __builtin_nontemporal_load(reinterpret_cast<const typename Raw4<ST>::type *>(p));
}
template <typename ST>
__device__ __forceinline__ void st_state4(ST *p, const float (&v)[4])
{
    typename Raw4<ST>::type w;
    if constexpr (sizeof(ST) == 4) {
        w = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    } else {
        uint16_t e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            put<ST>(&e[j], v[j]);
        w = u32x2{e[0] | ((uint32_t)e[1] << 16), e[2] | ((uint32_t)e[3] << 16)};
    }
    __builtin_nontemporal_store(w, reinterpret_cast<typename Raw4<ST>::type *>(p));
}

template <int W>
__device__ __forceinline__ float lanes_sum(float v)
{
    if constexpr (W == 2)
        return v + dpp_f32<0xB1>(v);  // quad_perm [1,0,3,2]
    else if constexpr (W >= 4 && W <= 16)
        return row_group_sum<W>(v);
    else if constexpr (W > 16)
        return group_sum<W>(v);
    return v;
}

// One token at a time; a thread has P channels, CH apart, which amortises the
// wave's start over more state. IO, DT, BC: element sizes of x/z/out, dt and B/C
// (0: any).
template <typename ST, int LPC, int P, int IO, int DT, int BC>
__global__ __launch_bounds__(256) void ssu_scan_rows_kernel(const ScanParams p, int tiles)
{
    constexpr int CH = 256 / LPC;  // channels of a workgroup's pass
    const int sub = threadIdx.x & (LPC - 1);
    const int b = blockIdx.x / tiles;
    const int first = (blockIdx.x - b * tiles) * (CH * P) + threadIdx.x / LPC;
    // lanes past the last channel repeat it, lanes past dstate the last four
    // entries (and count for nothing)
    const int n0 = min(sub * 4, p.dstate - 4);
    const bool own = sub * 4 < p.dstate;
    int row;
    const int len = row_tokens(p, b, &row);
    int d[P];
#pragma unroll
    for (int i = 0; i < P; ++i)
        d[i] = min(first + i * CH, p.dim - 1);
    if (len == 0) {
        if (p.out && sub == 0) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (first + i * CH < p.dim)
                    st1<IO>(p.out, b * p.out_bs + d[i], 0.0f, p.io_dtype);
        }
        return;
    }
    // absent operands are loaded from a present one and not used
    const void *zsrc = p.z ? p.z : p.x, *csrc = p.out ? p.C : p.B;
    const int64_t zb = p.z ? b * p.z_bs : b * p.x_bs, cb = p.out ? b * p.c_bs : b * p.b_bs;
    const float *bsrc = p.dt_bias ? p.dt_bias : p.A, *dsrc = p.D ? p.D : p.A;
    ST *st = static_cast<ST *>(p.state) + (int64_t)row * p.row_stride + n0;
    typename Raw4<ST>::type hraw[P];
    int64_t bc[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        hraw[i] = ld_state4<ST>(st + (int64_t)d[i] * p.dstate);
        bc[i] = (p.ngroups == 1 ? 0 : d[i] / (p.dim / p.ngroups)) * (int64_t)p.dstate + n0;
    }
    uint32_t x[P], dt[P], z[P];
    Raw4x rb[P], rc[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        dt[i] = raw1<DT>(p.dt, b * p.dt_bs + d[i], p.dt_dtype);
        x[i] = raw1<IO>(p.x, b * p.x_bs + d[i], p.io_dtype);
        z[i] = raw1<IO>(zsrc, zb + d[i], p.io_dtype);
        rb[i] = raw4<BC>(p.B, b * p.b_bs + bc[i], p.bc_dtype);
        rc[i] = raw4<BC>(csrc, cb + bc[i], p.bc_dtype);
    }
    float4 aw[P];
    float bias[P], skip[P], h[P][4];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        aw[i] = *reinterpret_cast<const float4 *>(p.A + (int64_t)d[i] * p.dstate + n0);
        bias[i] = bsrc[d[i]];
        skip[i] = dsrc[d[i]];
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        bias[i] = p.dt_bias ? bias[i] : 0.0f;
        skip[i] = p.D ? skip[i] : 0.0f;
        cvt_raw4<ST>(hraw[i], h[i]);
    }
    float v[P], y[P];
#pragma unroll
    for (int i = 0; i < P; ++i)
        v[i] = cvt1<DT>(dt[i], p.dt_dtype) + bias[i];
    if (p.dt_softplus) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            v[i] = softplus_f32(v[i]);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float xv = cvt1<IO>(x[i], p.io_dtype), u = v[i] * xv;
        const float a[4] = {log2_rate(aw[i].x), log2_rate(aw[i].y), log2_rate(aw[i].z), log2_rate(aw[i].w)};
        float bv[4], cv[4], acc = 0.0f;
        cvt4<BC>(rb[i], p.bc_dtype, bv);
        cvt4<BC>(rc[i], p.bc_dtype, cv);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[i][j] = fmaf(h[i][j], __builtin_amdgcn_exp2f(a[j] * v[i]), u * bv[j]);
            acc = fmaf(h[i][j], cv[j], acc);
        }
        y[i] = fmaf(skip[i], xv, lanes_sum<LPC>(own ? acc : 0.0f));
    }
    if (p.out) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (p.z)
                y[i] *= silu_hw(cvt1<IO>(z[i], p.io_dtype));
            if (sub == 0 && first + i * CH < p.dim)
                st1<IO>(p.out, b * p.out_bs + d[i], y[i], p.io_dtype);
        }
    }
    if (p.update && own) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (first + i * CH < p.dim)
                st_state4<ST>(st + (int64_t)d[i] * p.dstate, h[i]);
    }
}

// The value of lane k of each quad, in all its lanes.
template <int K>
__device__ __forceinline__ float quad_lane(float v)
{
    return dpp_f32<K * 0x55>(v);  // quad_perm [K,K,K,K]
}

// A few tokens, four at a time: lane k of a quad has token t0 + k's x, dt and z,
// so that its loads, softplus, gate and store happen once and not on each of
// the channel's lanes; dt' and dt' x then go round the quad.
template <typename ST, int LPC, int IO, int DT, int BC>
__global__ __launch_bounds__(256) void ssu_scan_window_kernel(const ScanParams p, int tiles)
{
    constexpr int CH = 256 / LPC, K = 4;
    const int sub = threadIdx.x & (LPC - 1), mine = threadIdx.x & (K - 1);
    const int b = blockIdx.x / tiles;
    const int d_raw = (blockIdx.x - b * tiles) * CH + threadIdx.x / LPC;
    // lanes past the last channel repeat it, lanes past dstate the last four
    // entries (and count for nothing)
    const int d = min(d_raw, p.dim - 1);
    const int n0 = min(sub * 4, p.dstate - 4);
    const bool own = sub * 4 < p.dstate;
    int row;
    const int len = row_tokens(p, b, &row);
    const bool stores = p.out && sub < K && d_raw < p.dim;
    if (stores)
        for (int t = len + mine; t < p.seq_len; t += K)
            st1<IO>(p.out, b * p.out_bs + t * p.out_ts + d, 0.0f, p.io_dtype);
    if (len == 0)
        return;
    // absent operands are loaded from a present one and not used
    const void *zsrc = p.z ? p.z : p.x, *csrc = p.out ? p.C : p.B;
    const int64_t zb = p.z ? b * p.z_bs : b * p.x_bs, zt = p.z ? p.z_ts : p.x_ts;
    const int64_t cb = p.out ? b * p.c_bs : b * p.b_bs, ct = p.out ? p.c_ts : p.b_ts;
    const float *bsrc = p.dt_bias ? p.dt_bias : p.A, *dsrc = p.D ? p.D : p.A;
    ST *st = static_cast<ST *>(p.state) + (int64_t)row * p.row_stride + (int64_t)d * p.dstate + n0;
    const auto hraw = ld_state4<ST>(st);
    const int64_t bc = (p.ngroups == 1 ? 0 : d / (p.dim / p.ngroups)) * (int64_t)p.dstate + n0;
    uint32_t x, dt, z;
    Raw4x rb[K], rc[K];
    auto load = [&](int t0) {
        const int t = min(t0 + mine, len - 1);
        dt = raw1<DT>(p.dt, b * p.dt_bs + t * p.dt_ts + d, p.dt_dtype);
        x = raw1<IO>(p.x, b * p.x_bs + t * p.x_ts + d, p.io_dtype);
        z = raw1<IO>(zsrc, zb + t * zt + d, p.io_dtype);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (t0 + k < len) {
                rb[k] = raw4<BC>(p.B, b * p.b_bs + (t0 + k) * p.b_ts + bc, p.bc_dtype);
                rc[k] = raw4<BC>(csrc, cb + (t0 + k) * ct + bc, p.bc_dtype);
            }
    };
    load(0);
    const float4 aw = *reinterpret_cast<const float4 *>(p.A + (int64_t)d * p.dstate + n0);
    float bias = bsrc[d], skip = dsrc[d], h[4];
    bias = p.dt_bias ? bias : 0.0f;
    skip = p.D ? skip : 0.0f;
    const float a[4] = {log2_rate(aw.x), log2_rate(aw.y), log2_rate(aw.z), log2_rate(aw.w)};
    cvt_raw4<ST>(hraw, h);
    for (int t0 = 0; t0 < len; t0 += K) {
        float v = cvt1<DT>(dt, p.dt_dtype) + bias;
        const float xv = cvt1<IO>(x, p.io_dtype), zv = cvt1<IO>(z, p.io_dtype);
        float bv[K][4], cv[K][4];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            cvt4<BC>(rb[k], p.bc_dtype, bv[k]);
            cvt4<BC>(rc[k], p.bc_dtype, cv[k]);
        }
        if (t0 + K < len)
            load(t0 + K);
        if (p.dt_softplus)
            v = softplus_f32(v);
        const float u = v * xv;
        float y = 0.0f;
        auto token = [&](auto kk) {
            constexpr int k = decltype(kk)::value;
            if (t0 + k >= len)
                return;
            float acc = 0.0f;
            const float vk = quad_lane<k>(v), uk = quad_lane<k>(u);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = fmaf(h[j], __builtin_amdgcn_exp2f(a[j] * vk), uk * bv[k][j]);
                acc = fmaf(h[j], cv[k][j], acc);
            }
            acc = lanes_sum<LPC>(own ? acc : 0.0f);
            y = mine == k ? acc : y;
        };
        token(std::integral_constant<int, 0>());
        token(std::integral_constant<int, 1>());
        token(std::integral_constant<int, 2>());
        token(std::integral_constant<int, 3>());
        if (stores && t0 + mine < len) {
            y = fmaf(skip, xv, y);
            if (p.z)
                y *= silu_hw(zv);
            st1<IO>(p.out, b * p.out_bs + (t0 + mine) * p.out_ts + d, y, p.io_dtype);
        }
    }
    if (p.update && own && d_raw < p.dim)
        st_state4<ST>(st, h);
}

template <typename Kernel>
hipError_t launch_tiles(Kernel kernel, const ScanParams &p, int channels, hipStream_t stream)
{
    const int tiles = (p.dim + channels - 1) / channels;
    const int64_t blocks = (int64_t)p.batch * tiles;
    if (!launchable(blocks, 256))
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, stream, p, tiles);
    return hipGetLastError();
}

template <typename ST, int LPC, int IO, int DT, int BC>
hipError_t launch_rows_types(const ScanParams &p, hipStream_t stream)
{
    constexpr int CH = 256 / LPC;
    if (p.seq_len > 1)
        return launch_tiles(ssu_scan_window_kernel<ST, LPC, IO, DT, BC>, p, CH, stream);
    // two channels a thread once that leaves two workgroups for every CU
    // (64 x 5120, dstate 16: 12.6 us, one 13.2, four 12.8)
    if (IO != 0 && (int64_t)p.batch * p.dim * LPC >= (int64_t)1024 * 256)
        return launch_tiles(ssu_scan_rows_kernel<ST, LPC, 2, IO, DT, BC>, p, 2 * CH, stream);
    return launch_tiles(ssu_scan_rows_kernel<ST, LPC, 1, IO, DT, BC>, p, CH, stream);
}

// 16-bit activations with dt in 16 or 32 bits, and everything in 32, have
// kernels of their own where B and C can be read four at a time.
template <typename ST, int LPC>
hipError_t launch_rows(const ScanParams &p, hipStream_t stream)
{
    const bool io4 = p.io_dtype == kF32, dt4 = p.dt_dtype == kF32, bc4 = p.bc_dtype == kF32;
    auto vec = [&](const void *q, int64_t bs, int64_t ts) {
        return (uintptr_t)q % (bc4 ? 16 : 8) == 0 && bs % 4 == 0 && ts % 4 == 0;
    };
    if (io4 == bc4 && vec(p.B, p.b_bs, p.b_ts) && (!p.out || vec(p.C, p.c_bs, p.c_ts))) {
        if (!io4 && !dt4)
            return launch_rows_types<ST, LPC, 2, 2, 2>(p, stream);
        if (!io4)
            return launch_rows_types<ST, LPC, 2, 4, 2>(p, stream);
        if (dt4)
            return launch_rows_types<ST, LPC, 4, 4, 4>(p, stream);
    }
    return launch_rows_types<ST, LPC, 0, 0, 0>(p, stream);
}

template <typename ST>
hipError_t launch_rows_lanes(const ScanParams &p, hipStream_t stream)
{
    if (p.dstate <= 16) return launch_rows<ST, 4>(p, stream);
    if (p.dstate <= 32) return launch_rows<ST, 8>(p, stream);
    if (p.dstate <= 64) return launch_rows<ST, 16>(p, stream);
    if (p.dstate <= 128) return launch_rows<ST, 32>(p, stream);
    return launch_rows<ST, 64>(p, stream);
}

}  // namespace

hipError_t launch_scan_rows(const ScanParams &p, hipStream_t stream)
{
    switch (p.state_dtype) {
    case kF32: return launch_rows_lanes<float>(p, stream);
    case kF16: return launch_rows_lanes<_Float16>(p, stream);
    default: return launch_rows_lanes<bf16_t>(p, stream);
    }
}

}  // namespace ssu
