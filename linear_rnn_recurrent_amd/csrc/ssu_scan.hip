// Per-channel selective scan over a paged state pool, for prompts and single
// tokens:
//   dt' = dt + dt_bias (softplus);  h[d,n] = h[d,n] exp(A[d,n] dt') + B[n] dt' x[d]
//   out[d] = (sum_n h[d,n] C[n] + D[d] x[d]) silu(z[d])
//
// Two evaluations, by the number of tokens (scan_plan):
//
// Rows (single tokens, windows of a few tokens): LPC lanes share a channel, four
// state entries each, so that the state, all but a few percent of the bytes, is
// read and written in whole cache lines; the sum over dstate is a butterfly
// across the channel's lanes. Bound by HBM.
//
// Chunks (prompts): the vector ALU bounds these (per token, channel and state
// entry a product, an exponential at half rate, a product and two fused
// multiply-adds: 6 issue slots), so the layout spends nothing else on the
// state entries: a lane is a channel and holds 16 state entries, which makes B and C the same
// for the whole wave (scalar registers, no lane traffic) and the sum over
// dstate private to the lane. One sequence has too few channels to fill the
// GPU that way, so its tokens are cut into chunks that run side by side:
//   pack    B and C of every token in fp32, padded to 16 states (scalar loads)
//   ends    every chunk's state from a zero start, and its sum of dt'
//           (the chunk's decay is exp(A sum dt'))
//   tokens  every chunk's start from the pool's state and the ends before it, in
//           order, then its tokens: the outputs, the last state
// (a single chunk needs no ends; without outputs a small kernel folds the ends
// into the last state and the tokens are not run)
// The chunks' decays are computed twice (11 slots instead of 6), against 1/16
// of the SIMDs busy without the cut at one sequence of 5,120 channels. dstate
// above 16 takes ceil(dstate / 16) waves, whose partial outputs meet in LDS.
#include <atomic>
#include <type_traits>
#include <utility>

#include "ssu_device.h"
#include "ssu_dpp.h"
#include "ssu_internal.h"

namespace ssu {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kStates = 16;  // state entries of a lane in the chunk kernels
constexpr int kBatch = 4;    // tokens loaded together

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

__device__ __forceinline__ int row_tokens(const ScanParams &p, int b, int *row)
{
    *row = p.idx ? p.idx[b] : b;
    return *row < 0 ? 0 : (p.ctx ? clamp_len(p.ctx[b], p.seq_len) : p.seq_len);
}

// ---------------------------------------------------------------------------
// Rows: LPC lanes per channel
// ---------------------------------------------------------------------------
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
        const float a[4] = {aw[i].x * kLog2e, aw[i].y * kLog2e, aw[i].z * kLog2e, aw[i].w * kLog2e};
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
    const float a[4] = {aw.x * kLog2e, aw.y * kLog2e, aw.z * kLog2e, aw.w * kLog2e};
    cvt_raw4<ST>(hraw, h);
    for (int t0 = 0; t0 < len; t0 += K) {
        float v = cvt1<DT>(dt, p.dt_dtype) + bias;
        if (p.dt_softplus)
            v = softplus_f32(v);
        const float xv = cvt1<IO>(x, p.io_dtype), zv = cvt1<IO>(z, p.io_dtype);
        const float u = v * xv;
        float y = 0.0f;
        auto token = [&](auto kk) {
            constexpr int k = decltype(kk)::value;
            if (t0 + k >= len)
                return;
            float bv[4], cv[4], acc = 0.0f;
            cvt4<BC>(rb[k], p.bc_dtype, bv);
            cvt4<BC>(rc[k], p.bc_dtype, cv);
            const float vk = quad_lane<k>(v), uk = quad_lane<k>(u);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = fmaf(h[j], __builtin_amdgcn_exp2f(a[j] * vk), uk * bv[j]);
                acc = fmaf(h[j], cv[j], acc);
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
        if (t0 + K < len)
            load(t0 + K);
    }
    if (p.update && own && d_raw < p.dim)
        st_state4<ST>(st, h);
}

template <typename Kernel>
hipError_t launch_tiles(Kernel kernel, const ScanParams &p, int channels, hipStream_t stream)
{
    const int tiles = (p.dim + channels - 1) / channels;
    const int64_t blocks = (int64_t)p.batch * tiles;
    if (blocks > 0x7fffffff)
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

// ---------------------------------------------------------------------------
// Chunks
// ---------------------------------------------------------------------------
// Workspace, in floats: packed B | C [batch][seq_len][ngroups][tiles][2][16],
// and a line of 32 zeros; chunk ends [batch][chunks + 1][blocks][tiles][16][64]
// (slot 0 a copy of the pool's state, so that the kernel that writes the pool
// does not read it; slot c + 1 chunk c's end); chunk sums of dt'
// [batch][chunks + 1][blocks][64], slot c + 1 likewise. A block is 64 channels
// of one group.
struct ChunkShape {
    int32_t tiles, per_group, blocks, chunk, chunks;
    int32_t team;  // chunks of one block that share a workgroup: 1, 2 or 4
    int64_t zeros;  // offset of the zero line in bc
    float *bc, *start, *sum;
};

// The block of channels, the batch row and the team of chunks of a workgroup.
struct Place {
    int b, team, blk, g, d, dl;  // .., group, channel (clamped), whether its lane is live
};

__device__ __forceinline__ Place place(const ScanParams &p, const ChunkShape &s, int teams)
{
    Place q;
    int i = blockIdx.x;
    q.blk = i % s.blocks;
    i /= s.blocks;
    q.team = i % teams;
    q.b = i / teams;
    q.g = q.blk / s.per_group;
    const int width = p.dim / p.ngroups;
    const int local = (q.blk - q.g * s.per_group) * 64 + (int)(threadIdx.x & 63);
    q.dl = local < width;
    q.d = q.g * width + min(local, width - 1);
    return q;
}

// B and C in fp32 (C's half is not written without outputs).
__global__ __launch_bounds__(256) void ssu_scan_pack_kernel(const ScanParams p, const ChunkShape s,
                                                            int64_t total)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (blockIdx.x == 0 && threadIdx.x < 2 * kStates)
        s.bc[s.zeros + threadIdx.x] = 0.0f;
    if (i >= total)
        return;
    const int n16 = s.tiles * kStates;
    const int n = (int)(i % n16);
    int64_t r = i / n16;
    const int g = (int)(r % p.ngroups);
    r /= p.ngroups;
    const int t = (int)(r % p.seq_len);
    const int b = (int)(r / p.seq_len);
    int row;
    if (t >= row_tokens(p, b, &row))
        return;
    float *o = s.bc + (i / kStates) * (2 * kStates) + (n & (kStates - 1));
    const bool in = n < p.dstate;
    const int64_t e = (int64_t)g * p.dstate + n;
    o[0] = in ? ld_io(p.B, b * p.b_bs + t * p.b_ts + e, p.bc_dtype) : 0.0f;
    if (p.out)
        o[kStates] = in ? ld_io(p.C, b * p.c_bs + t * p.c_ts + e, p.bc_dtype) : 0.0f;
}

// A[d, 16 tile ..] log2(e); entries past dstate are 0.
__device__ __forceinline__ void load_a(const ScanParams &p, int d, int tile, float (&a)[kStates])
{
#pragma unroll
    for (int j = 0; j < kStates; j += 4) {
        float4 w = make_float4(0, 0, 0, 0);
        if (tile * kStates + j < p.dstate)
            w = *reinterpret_cast<const float4 *>(p.A + (int64_t)d * p.dstate + tile * kStates + j);
        a[j] = w.x * kLog2e;
        a[j + 1] = w.y * kLog2e;
        a[j + 2] = w.z * kLog2e;
        a[j + 3] = w.w * kLog2e;
    }
}

// One activation [.., seq_len, dim] read a batch of tokens at a time: a scalar
// base that moves by batches, and a byte offset per token of the batch and lane,
// so that a load costs no address arithmetic. (Host: 4 token strides < 2^31 bytes.)
template <typename T>
struct Stream {
    static constexpr int SZ = sizeof(T) == 4 ? 4 : 2;
    using E = typename std::conditional<SZ == 4, uint32_t, uint16_t>::type;
    const char *base;
    int64_t step;
    uint32_t off[kBatch];

    __device__ __forceinline__ Stream(const void *p, int64_t first, int64_t ts, int d)
        : base(static_cast<const char *>(p) + first * SZ), step(ts * (kBatch * SZ))
    {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            off[i] = (uint32_t)(i * ts * SZ) + (uint32_t)d * SZ;
    }
    // `n` tokens are left: the ones past them read the last of them
    __device__ __forceinline__ void load(int n, uint32_t (&w)[kBatch])
    {
        if (n < kBatch) {
#pragma unroll
            for (int i = 1; i < kBatch; ++i)
                off[i] = i < n ? off[i] : off[i - 1];
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            w[i] = *reinterpret_cast<const E *>(base + off[i]);
        base += step;
    }
};

// dt' and dt' x of a batch; tokens from `n` on are neutral (dt' = 0 leaves the
// state as it is), so that every batch runs the same straight code.
template <typename IOT, typename DTT>
__device__ __forceinline__ void step_sizes(const uint32_t (&x)[kBatch], const uint32_t (&dt)[kBatch],
                                           float bias, bool softplus, int n, float (&v)[kBatch],
                                           float (&u)[kBatch])
{
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
        v[i] = cvt_raw1<DTT>(dt[i]) + bias;
    if (softplus) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            v[i] = softplus_f32(v[i]);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        v[i] = i < n ? v[i] : 0.0f;
        u[i] = i < n ? v[i] * cvt_raw1<IOT>(x[i]) : 0.0f;
    }
}

// Every chunk's end from a zero start (all but a row's last chunk, or all of
// them where only the state is wanted), and the copy of the pool's state.
template <typename IOT, typename DTT>
__global__ __launch_bounds__(256, 4) void ssu_scan_ends_kernel(const ScanParams p,
                                                               const ChunkShape s,
                                                               const float *__restrict__ packed)
{
    const Place q = place(p, s, (s.chunks + s.team - 1) / s.team);
    const int c = q.team * s.team + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile = blockIdx.y;
    const int lane = threadIdx.x & 63;
    int row;
    const int len = row_tokens(p, q.b, &row);
    const int t0 = c * s.chunk, t1 = min(t0 + s.chunk, len);
    const int64_t at = ((int64_t)q.b * (s.chunks + 1) + c) * s.blocks + q.blk;
    float *e = s.start + (at * s.tiles + tile) * (kStates * 64) + lane;
    if (t0 >= len)
        return;
    if (c == 0) {
        const int64_t so = (int64_t)row * p.row_stride + (int64_t)q.d * p.dstate + tile * kStates;
#pragma unroll
        for (int j = 0; j < kStates; ++j)
            e[j * 64] = tile * kStates + (j & ~3) < p.dstate ? ld_io(p.state, so + j, p.state_dtype)
                                                              : 0.0f;
    }
    if (p.out && t1 == len)
        return;
    e += (int64_t)s.blocks * s.tiles * (kStates * 64);
    const int64_t bc_step = (int64_t)p.ngroups * s.tiles * 2 * kStates;
    int64_t bc = ((((int64_t)q.b * p.seq_len + t0) * p.ngroups + q.g) * s.tiles + tile) * (2 * kStates);
    const float bias = p.dt_bias ? p.dt_bias[q.d] : 0.0f;
    Stream<IOT> xs(p.x, q.b * p.x_bs + t0 * p.x_ts, p.x_ts, q.d);
    Stream<DTT> ds(p.dt, q.b * p.dt_bs + t0 * p.dt_ts, p.dt_ts, q.d);
    float a[kStates], h[kStates] = {}, sum = 0.0f;
    uint32_t x[kBatch], dt[kBatch];
    xs.load(t1 - t0, x);
    ds.load(t1 - t0, dt);
    load_a(p, q.d, tile, a);
    float bs[kStates];  // the next token's B
#pragma unroll
    for (int j = 0; j < kStates; ++j)
        bs[j] = packed[bc + j];
    for (int t = t0; t < t1; t += kBatch) {
        float v[kBatch], u[kBatch];
        step_sizes<IOT, DTT>(x, dt, bias, p.dt_softplus, t1 - t, v, u);
        if (t + kBatch < t1) {
            xs.load(t1 - t - kBatch, x);
            ds.load(t1 - t - kBatch, dt);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            bc = t + i + 1 < t1 ? bc + bc_step : s.zeros;
            float bn[kStates];
#pragma unroll
            for (int j = 0; j < kStates; ++j)
                bn[j] = packed[bc + j];
            sum += v[i];
#pragma unroll
            for (int j = 0; j < kStates; ++j) {
                h[j] = fmaf(h[j], __builtin_amdgcn_exp2f(a[j] * v[i]), u[i] * bs[j]);
                bs[j] = bn[j];
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int j = 0; j < kStates; ++j)
        e[j * 64] = h[j];
    if (tile == 0)
        s.sum[(at + s.blocks) * 64 + lane] = sum;
}

// Runs the starts of chunks first, first + 1, .. of NS state entries (from j0
// of a tile) through the ends in order: use(c, h) sees the start of chunk c for
// c = from .. to.
template <int NS, typename Use>
__device__ __forceinline__ void fold_ends(const ScanParams &p, const ChunkShape &s, const Place &q,
                                          int tile, int j0, int from, int to, Use use)
{
    const int64_t step = (int64_t)s.blocks * s.tiles * (kStates * 64), sum_step = s.blocks * 64;
    const int64_t first = (int64_t)q.b * (s.chunks + 1) * s.blocks + q.blk;
    const float *e = s.start + (first * s.tiles + tile) * (kStates * 64) + j0 * 64 + (threadIdx.x & 63);
    const float *sum = s.sum + first * 64 + (threadIdx.x & 63);
    float a[NS], h[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int n = tile * kStates + j0 + j;
        a[j] = n < p.dstate ? p.A[(int64_t)q.d * p.dstate + n] * kLog2e : 0.0f;
        h[j] = e[j * 64];
    }
    constexpr int F = 32 / NS;  // ends in flight
    for (int c = 0; c < to; c += F) {
        float end[F][NS], total[F];
#pragma unroll
        for (int i = 0; i < F; ++i) {
            const int k = min(c + i, to - 1) + 1;
            total[i] = sum[k * sum_step];
#pragma unroll
            for (int j = 0; j < NS; ++j)
                end[i][j] = e[k * step + j * 64];
        }
#pragma unroll
        for (int i = 0; i < F; ++i) {
            if (c + i < to) {
                if (c + i >= from)
                    use(c + i, h);
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    h[j] = fmaf(h[j], __builtin_amdgcn_exp2f(a[j] * total[i]), end[i][j]);
            }
        }
    }
    use(to, h);
}

// The last state where no outputs are wanted; a wave has one state entry of a
// tile.
__global__ __launch_bounds__(1024) void ssu_scan_last_kernel(const ScanParams p, const ChunkShape s)
{
    const Place q = place(p, s, 1);
    const int tile = blockIdx.y;
    int row;
    const int len = row_tokens(p, q.b, &row);
    if (len == 0)
        return;
    const int j0 = threadIdx.x >> 6, n0 = tile * kStates + j0;
    const int chunks = (len + s.chunk - 1) / s.chunk;
    fold_ends<1>(p, s, q, tile, j0, chunks, chunks, [&](int, const float (&h)[1]) {
        if (p.update && n0 < p.dstate && q.dl)
            st_io(p.state, (int64_t)row * p.row_stride + (int64_t)q.d * p.dstate + n0, h[0],
                  p.state_dtype);
    });
}

// The tokens of a team of chunks: tiles waves a chunk, one per 16 state
// entries. The team's waves first share the fold of the ends before it (each
// folds its part of every tile's entries; the starts meet in LDS). With more
// than one tile a batch's partial outputs are summed through LDS (two buffers,
// so one barrier a batch) and its tokens finished by the chunk's waves in turn.
template <typename IOT, typename DTT, bool ONE>
__global__ __launch_bounds__(ONE ? 256 : 1024, 4) void ssu_scan_tokens_kernel(
    const ScanParams p, const ChunkShape s, const float *__restrict__ packed,
    void *__restrict__ out)
{
    // [team][tiles][16][64] starts, then unless ONE [2][team][tiles][kBatch][64]
    extern __shared__ float lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile = ONE ? 0 : wave % s.tiles;
    const int mate = ONE ? wave : wave / s.tiles;
    const Place q = place(p, s, (s.chunks + s.team - 1) / s.team);
    const int c0 = q.team * s.team, c = c0 + mate;
    int row;
    const int len = row_tokens(p, q.b, &row);
    const int t0 = c * s.chunk, t_end = min(t0 + s.chunk, p.seq_len), t1 = min(t_end, len);
    // lanes past the last channel repeat it: they store the same values
    constexpr int SZ = Stream<IOT>::SZ;
    char *o = static_cast<char *>(out) + (q.b * p.out_bs + t0 * p.out_ts) * SZ;
    uint32_t off[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
        off[i] = (uint32_t)(i * p.out_ts * SZ) + (uint32_t)q.d * SZ;
    for (int t = max(t0, len) + tile; t < t_end; t += ONE ? 1 : s.tiles)
        put<IOT>(o + (t - t0) * p.out_ts * SZ + off[0], 0.0f);
    if (c0 * s.chunk >= len)  // the whole team
        return;

    const bool live = t0 < len;
    const int64_t bc_step = (int64_t)p.ngroups * s.tiles * 2 * kStates;
    int64_t bc = ((((int64_t)q.b * p.seq_len + t0) * p.ngroups + q.g) * s.tiles + tile) * (2 * kStates);
    const float bias = p.dt_bias ? p.dt_bias[q.d] : 0.0f;
    const float skip = p.D ? p.D[q.d] : 0.0f;
    const int64_t so = (int64_t)row * p.row_stride + (int64_t)q.d * p.dstate + tile * kStates;
    const bool gated = p.z != nullptr;  // without a gate x is loaded in z's place and not used
    Stream<IOT> xs(p.x, q.b * p.x_bs + t0 * p.x_ts, p.x_ts, q.d);
    Stream<IOT> zs(gated ? p.z : p.x, gated ? q.b * p.z_bs + t0 * p.z_ts : q.b * p.x_bs + t0 * p.x_ts,
                   gated ? p.z_ts : p.x_ts, q.d);
    Stream<DTT> ds(p.dt, q.b * p.dt_bs + t0 * p.dt_ts, p.dt_ts, q.d);
    uint32_t x[kBatch], dt[kBatch], z[kBatch];
    auto load = [&](int n) {
        xs.load(n, x);
        ds.load(n, dt);
        zs.load(n, z);
    };
    if (live)
        load(t1 - t0);
    float a[kStates], h[kStates] = {};
    load_a(p, q.d, tile, a);
    if (s.chunks > 1) {
        // the team's last chunk with tokens
        const int to = min(c0 + s.team, (len + s.chunk - 1) / s.chunk) - 1;
        auto share = [&](auto ns) {
            constexpr int NS = decltype(ns)::value;
            const int j0 = mate * NS;
            fold_ends<NS>(p, s, q, tile, j0, c0, to, [&](int k, const float (&st)[NS]) {
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    lds[(((k - c0) * s.tiles + tile) * kStates + j0 + j) * 64 + lane] = st[j];
            });
        };
        if (s.team == 4)
            share(std::integral_constant<int, 4>());
        else if (s.team == 2)
            share(std::integral_constant<int, 8>());
        else
            share(std::integral_constant<int, 16>());
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kStates; ++j)
            h[j] = lds[((mate * s.tiles + tile) * kStates + j) * 64 + lane];
    } else {
#pragma unroll
        for (int j = 0; j < kStates; ++j)
            if (tile * kStates + (j & ~3) < p.dstate)
                h[j] = ld_io(p.state, so + j, p.state_dtype);
    }
    if (ONE && !live)
        return;
    // the batches of the team's first chunk, the longest (every wave meets the
    // barriers)
    const int batches = (min(s.chunk, len - (ONE ? t0 : c0 * s.chunk)) + kBatch - 1) / kBatch;
    float *part = lds + (s.chunks > 1 ? s.team * s.tiles * kStates * 64 : 0);
    if (!live)
        bc = s.zeros;
    float bs[kStates];  // the next token's B
#pragma unroll
    for (int j = 0; j < kStates; ++j)
        bs[j] = packed[bc + j];
    int buf = 0;
    for (int t = t0; t < t0 + batches * kBatch; t += kBatch) {
        if (!ONE && t >= t1) {
            __syncthreads();
            continue;
        }
        float v[kBatch], u[kBatch], sk[kBatch], gate[kBatch], y[kBatch];
        step_sizes<IOT, DTT>(x, dt, bias, p.dt_softplus, t1 - t, v, u);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            sk[i] = skip * cvt_raw1<IOT>(x[i]);
            gate[i] = cvt_raw1<IOT>(z[i]);
        }
        if (t + kBatch < t1)
            load(t1 - t - kBatch);
        // token i's C and token i + 1's B (scalar loads) are on their way while
        // token i's states are computed; the barriers keep that order
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            float cs[kStates], bn[kStates];
#pragma unroll
            for (int j = 0; j < kStates; ++j)
                cs[j] = packed[bc + kStates + j];
            bc = t + i + 1 < t1 ? bc + bc_step : s.zeros;
#pragma unroll
            for (int j = 0; j < kStates; ++j)
                bn[j] = packed[bc + j];
#pragma unroll
            for (int j = 0; j < kStates; ++j)
                h[j] = fmaf(h[j], __builtin_amdgcn_exp2f(a[j] * v[i]), u[i] * bs[j]);
            __builtin_amdgcn_sched_barrier(0);
            float y2[2] = {0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < kStates; ++j) {
                y2[j & 1] = fmaf(h[j], cs[j], y2[j & 1]);
                bs[j] = bn[j];
            }
            y[i] = y2[0] + y2[1];
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (!ONE) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                part[(((buf * s.team + mate) * s.tiles + tile) * kBatch + i) * 64 + lane] = y[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                y[i] = 0.0f;
                if (i % s.tiles == tile)
                    for (int k = 0; k < s.tiles; ++k)
                        y[i] += part[(((buf * s.team + mate) * s.tiles + k) * kBatch + i) * 64 + lane];
            }
            buf ^= 1;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            y[i] += sk[i];
        if (gated) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                y[i] *= silu_hw(gate[i]);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (t + i < t1 && (ONE || i % s.tiles == tile))
                put<IOT>(o + off[i], y[i]);
        o += p.out_ts * (kBatch * SZ);
    }
    if (p.update && live && t1 == len) {
#pragma unroll
        for (int j = 0; j < kStates; ++j)
            if (tile * kStates + (j & ~3) < p.dstate)
                st_io(p.state, so + j, h[j], p.state_dtype);
    }
}

// ---------------------------------------------------------------------------
// Sweep
// ---------------------------------------------------------------------------
constexpr int kSub = 16;             // tokens of a wave's part of a step
constexpr int kSweepWaves = 8;
constexpr int kSweep = kSub * kSweepWaves;  // tokens of a step
constexpr int kVuPitch = 2 * kSub + 4;      // floats: the 16 channels' rows 4 banks apart

template <typename F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>()), ...);
}

// Lane I of each row of 16, in all of the row's lanes.
template <int I>
__device__ __forceinline__ float row_lane(float v)
{
    const int u = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(u, u, 0x150 + I, 0xF, 0xF, true));
}

// Four adjacent B or C entries of one token as floats.
template <int BC>
__device__ __forceinline__ void ld_bc4(const char *base, uint32_t off, int dt, float (&v)[4])
{
    if constexpr (BC == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = cvt1<0>(raw1<0>(base + off, j, dt), dt);
    } else {
        cvt4<BC>(raw4<BC>(base + off, 0, dt), dt, v);
    }
}

// A workgroup sweeps 16 channels through a row's tokens, 128 a step. Lane (r, c)
// of a wave has four state entries (4r ..) of channel c and the wave 16 of the
// step's tokens: it runs them from a zero start keeping the 16 decays of each
// entry, the waves exchange ends and decays through LDS, and every wave runs its
// tokens again from its true start without any exponential. A token's B and C
// lie across the 16 lanes of a row and reach its channels by DPP broadcast; its
// dt' and dt' x go through the wave's own LDS; the sum over dstate is two
// swap-and-adds that also hand lane (r, c) the outputs of tokens 4r .. 4r + 3,
// whose x, dt and z it loaded. dstate above 16 repeats the two runs per 16.
template <typename IOT, typename DTT, int BC>
__global__ __launch_bounds__(64 * kSweepWaves, 4) void ssu_scan_sweep_kernel(
    const ScanParams p, int per_group, int blocks, int tiles)
{
    extern __shared__ float lds[];
    // [waves][16][kVuPitch] dt', dt' x; [2][waves][64][8] ends and decays; [2][tiles][64][4] states
    const int lane = threadIdx.x & 63, r = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float *vu = lds + wave * (16 * kVuPitch);
    float4 *ends = reinterpret_cast<float4 *>(lds + kSweepWaves * 16 * kVuPitch);
    float4 *starts = ends + 2 * kSweepWaves * 64 * 2;

    // eight neighbouring blocks, which share cache lines of x, dt, z and out, on
    // one XCD (workgroups go to the eight XCDs in turn)
    int id = blockIdx.x;
    if (id < (int)(gridDim.x & ~63u))
        id = (id & ~63) + (id & 7) * 8 + ((id >> 3) & 7);
    const int b = id / blocks, blk = id - b * blocks;
    const int g = blk / per_group;
    const int width = p.dim / p.ngroups;
    // lanes past the group's last channel repeat it: they store the same values
    const int d = g * width + min((blk - g * per_group) * 16 + c, width - 1);
    int row;
    const int len = row_tokens(p, b, &row);

    constexpr int SZ = sizeof(IOT) == 4 ? 4 : 2, DZ = sizeof(DTT) == 4 ? 4 : 2;
    using E = typename std::conditional<SZ == 4, uint32_t, uint16_t>::type;
    using DE = typename std::conditional<DZ == 4, uint32_t, uint16_t>::type;
    char *out = static_cast<char *>(p.out) + b * p.out_bs * SZ;
    const uint32_t dx = d * SZ, dd = d * DZ;
    if (p.out)
        for (int t = len + wave * 4 + r; t < p.seq_len; t += kSweepWaves * 4)
            put<IOT>(out + t * p.out_ts * SZ + dx, 0.0f);
    if (len == 0)
        return;

    const bool gated = p.z != nullptr;  // absent operands are loaded from a present one and not used
    const char *xp = static_cast<const char *>(p.x) + b * p.x_bs * SZ;
    const char *zp = gated ? static_cast<const char *>(p.z) + b * p.z_bs * SZ : xp;
    const int64_t zts = gated ? p.z_ts : p.x_ts;
    const char *dp = static_cast<const char *>(p.dt) + b * p.dt_bs * DZ;
    const int bz = p.bc_dtype == kF32 ? 4 : 2;
    const char *bp = static_cast<const char *>(p.B) + (b * p.b_bs + (int64_t)g * p.dstate) * bz;
    const char *cp = p.out ? static_cast<const char *>(p.C) + (b * p.c_bs + (int64_t)g * p.dstate) * bz : bp;
    const int64_t bts = p.b_ts * bz, cts = (p.out ? p.c_ts : p.b_ts) * bz;
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.0f;
    const float skip = p.D ? p.D[d] : 0.0f;
    const int64_t so = (int64_t)row * p.row_stride + (int64_t)d * p.dstate;

    // the states at the first step's start
    for (int k = wave; k < tiles; k += kSweepWaves) {
        float h[4] = {};
        const int n0 = k * kStates + r * 4;
        if (n0 < p.dstate) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                h[j] = ld_io(p.state, so + n0 + j, p.state_dtype);
        }
        starts[k * 64 + lane] = make_float4(h[0], h[1], h[2], h[3]);
    }
    int starts_now = 0;  // which of the two copies the step reads; the other gets the next's

    // a lane's byte offsets of its four tokens from the wave's first (host: 16
    // token strides < 2^32 bytes)
    const uint32_t xts = (uint32_t)p.x_ts * SZ, gts = (uint32_t)zts * SZ, dts = (uint32_t)p.dt_ts * DZ,
                   ots = (uint32_t)p.out_ts * SZ;
    E x[4], z[4];
    DE dt[4];
    auto load = [&](int t0) {  // this wave's tokens of the step at t0; past the row: its last
        const int w0 = min(t0 + wave * kSub, len - 1), most = len - 1 - w0;
        const char *xw = xp + w0 * p.x_ts * SZ, *zw = zp + w0 * zts * SZ, *dw = dp + w0 * p.dt_ts * DZ;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t t = min(r * 4 + q, most);
            x[q] = *reinterpret_cast<const E *>(xw + (t * xts + dx));
            z[q] = *reinterpret_cast<const E *>(zw + (t * gts + dx));
            dt[q] = *reinterpret_cast<const DE *>(dw + (t * dts + dd));
        }
    };
    load(0);
    int buf = 0;
    for (int t0 = 0; t0 < len; t0 += kSweep) {
        const int w0 = t0 + wave * kSub;  // the wave's first token
        float xs[4], gate[4], y4[4] = {};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v = cvt_raw1<DTT>(dt[q]) + bias;
            if (p.dt_softplus)
                v = softplus_f32(v);
            const bool in = w0 + r * 4 + q < len;  // others are neutral: dt' = 0
            v = in ? v : 0.0f;
            const float xv = cvt_raw1<IOT>(x[q]);
            *reinterpret_cast<float2 *>(vu + c * kVuPitch + (r * 4 + q) * 2) =
                make_float2(v, in ? v * xv : 0.0f);
            xs[q] = skip * xv;
            gate[q] = cvt_raw1<IOT>(z[q]);
        }
        __builtin_amdgcn_wave_barrier();
        if (t0 + kSweep < len)
            load(t0 + kSweep);
        for (int k = 0; k < tiles; ++k) {
            const int n0 = k * kStates + r * 4, nn = min(n0, p.dstate - 4);
            const bool own = n0 < p.dstate;
            const float4 aw = *reinterpret_cast<const float4 *>(p.A + (int64_t)d * p.dstate + nn);
            const int tok = min(w0 + c, len - 1);  // B and C: lane c has token c of the wave's
            float bv[4], cv[4];
            ld_bc4<BC>(bp + tok * bts, nn * bz, p.bc_dtype, bv);
            ld_bc4<BC>(cp + tok * cts, nn * bz, p.bc_dtype, cv);
            const float a[4] = {aw.x * kLog2e, aw.y * kLog2e, aw.z * kLog2e, aw.w * kLog2e};
            const bool real = own && w0 + c < len;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bv[j] = real ? bv[j] : 0.0f;
                cv[j] = real ? cv[j] : 0.0f;
            }
            // from a zero start
            float dec[kSub][4], h[4] = {}, sum = 0.0f;
            each_of(
                [&](auto tt) {
                    constexpr int t = decltype(tt)::value;
                    const float2 w = *reinterpret_cast<const float2 *>(vu + c * kVuPitch + t * 2);
                    sum += w.x;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        dec[t][j] = __builtin_amdgcn_exp2f(a[j] * w.x);
                        h[j] = fmaf(h[j], dec[t][j], row_lane<t>(bv[j]) * w.y);
                    }
                    __builtin_amdgcn_sched_barrier(0);  // keeps the tokens in order, and the registers few
                },
                std::make_integer_sequence<int, kSub>());
            float4 *mine = ends + ((buf * kSweepWaves + wave) * 64 + lane) * 2;
            mine[0] = make_float4(h[0], h[1], h[2], h[3]);
            mine[1] = make_float4(__builtin_amdgcn_exp2f(a[0] * sum), __builtin_amdgcn_exp2f(a[1] * sum),
                                  __builtin_amdgcn_exp2f(a[2] * sum), __builtin_amdgcn_exp2f(a[3] * sum));
            __syncthreads();
            // the wave's start
            const float4 s0 = starts[(starts_now * tiles + k) * 64 + lane];
            h[0] = s0.x, h[1] = s0.y, h[2] = s0.z, h[3] = s0.w;
            for (int m = 0; m < wave; ++m) {
                const float4 e = ends[((buf * kSweepWaves + m) * 64 + lane) * 2];
                const float4 f = ends[((buf * kSweepWaves + m) * 64 + lane) * 2 + 1];
                h[0] = fmaf(h[0], f.x, e.x);
                h[1] = fmaf(h[1], f.y, e.y);
                h[2] = fmaf(h[2], f.z, e.z);
                h[3] = fmaf(h[3], f.w, e.w);
            }
            buf ^= 1;
            float y[kSub];
            each_of(
                [&](auto tt) {
                    constexpr int t = decltype(tt)::value;
                    const float u = vu[c * kVuPitch + t * 2 + 1];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        h[j] = fmaf(h[j], dec[t][j], row_lane<t>(bv[j]) * u);
                        y[t] = j == 0 ? row_lane<t>(cv[j]) * h[j] : fmaf(row_lane<t>(cv[j]), h[j], y[t]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                },
                std::make_integer_sequence<int, kSub>());
            // sums over the four rows: halves, then rows, leaving tokens 4r .. 4r + 3
            float y8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(y[i]),
                                                                __float_as_uint(y[i + 8]), false, false);
                y8[i] = __uint_as_float(w[0]) + __uint_as_float(w[1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(y8[i]),
                                                                __float_as_uint(y8[i + 4]), false, false);
                y4[i] += __uint_as_float(w[0]) + __uint_as_float(w[1]);
            }
            if (wave == kSweepWaves - 1)
                starts[((starts_now ^ 1) * tiles + k) * 64 + lane] = make_float4(h[0], h[1], h[2], h[3]);
        }
        if (p.out) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v = y4[q] + xs[q];
                if (gated)
                    v *= silu_hw(gate[q]);
                if (w0 + r * 4 + q < len)
                    put<IOT>(out + w0 * p.out_ts * SZ + ((r * 4 + q) * ots + dx), v);
            }
        }
        starts_now ^= 1;
    }
    __syncthreads();
    if (p.update) {
        for (int k = wave; k < tiles; k += kSweepWaves) {
            const int n0 = k * kStates + r * 4;
            const float4 s0 = starts[(starts_now * tiles + k) * 64 + lane];
            const float h[4] = {s0.x, s0.y, s0.z, s0.w};
            if (n0 < p.dstate) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    st_io(p.state, so + n0 + j, h[j], p.state_dtype);
            }
        }
    }
}

// Which evaluation a call takes, and its cut. Chunks are as long as leaves about
// three waves for each of the GPU's 1,024 SIMDs: every chunk costs its end, its
// fold and 4 KiB of traffic, and too few leave SIMDs idle (1 x 2048 x 5120: 113 us
// at 2,560 waves, 102 at 3,072, 104 at 4,096, 109 at 8,192). With context_lengths
// rows end early and unevenly, and shorter chunks fill the gaps (8 x 777 x 2560
// with lengths from an eighth up: 135 us at 3,072, 93 at 6,144, 86 at 8,192, 87 at
// 10,000).
struct Plan {
    bool rows, sweep;
    ChunkShape s;
    int64_t bc_floats, start_floats, sum_floats;
};

Plan scan_plan(int64_t batch, int64_t dim, int64_t dstate, int64_t ngroups, int64_t seq_len,
               bool ragged)
{
    Plan q = {};
    q.rows = seq_len <= 16;
    if (q.rows)
        return q;
#ifndef SWEEP_MIN
#define SWEEP_MIN 192
#endif
    q.sweep = batch * ngroups * ((dim / ngroups + 15) / 16) >= SWEEP_MIN;
    if (q.sweep)
        return q;
    q.s.tiles = (int32_t)((dstate + kStates - 1) / kStates);
    q.s.per_group = (int32_t)((dim / ngroups + 63) / 64);
    q.s.blocks = (int32_t)(q.s.per_group * ngroups);
    const int64_t waves = batch * q.s.blocks * q.s.tiles, target = ragged ? 8192 : 3072;
    int64_t chunks = waves * 2 > target ? 1 : target / waves;
    int64_t len = (seq_len + chunks - 1) / chunks;
    len = (len + kBatch - 1) / kBatch * kBatch;
    if (len < 32)
        len = 32;
    chunks = (seq_len + len - 1) / len;
    q.s.chunk = (int32_t)(len > seq_len ? seq_len : len);
    q.s.chunks = (int32_t)chunks;
    const int most = q.s.tiles <= 4 ? 4 : q.s.tiles <= 8 ? 2 : 1;
    q.s.team = chunks == 1 ? 1 : (chunks == 2 && most > 2) ? 2 : most;
    q.bc_floats = (batch * seq_len * ngroups * q.s.tiles + 1) * (2 * kStates);
    q.start_floats = batch * (chunks + 1) * q.s.blocks * q.s.tiles * (kStates * 64);
    q.sum_floats = batch * (chunks + 1) * q.s.blocks * 64;
    return q;
}

// Dynamic LDS above the default 64 KiB is allowed once per kernel and device.
hipError_t raise_lds(const void *kernel, int bytes, std::atomic<uint64_t> *raised)
{
    if (bytes <= 65536)
        return hipSuccess;
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess || (dev < 64 && ((raised->load(std::memory_order_relaxed) >> dev) & 1)))
        return e;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 98304);
    if (e == hipSuccess && dev < 64)
        raised->fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

template <typename IOT, typename DTT>
hipError_t launch_chunks(const ScanParams &p, const Plan &q, hipStream_t stream)
{
    const ChunkShape &s = q.s;
    const int64_t cells = (int64_t)p.batch * s.blocks * ((s.chunks + s.team - 1) / s.team);
    const int64_t packed = q.bc_floats / 2 - kStates;
    if (cells > 0x7fffffff || (packed + 255) / 256 > 0x7fffffff)
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(ssu_scan_pack_kernel, dim3((unsigned)((packed + 255) / 256)), dim3(256), 0,
                       stream, p, s, packed);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && (s.chunks > 1 || !p.out)) {
        hipLaunchKernelGGL((ssu_scan_ends_kernel<IOT, DTT>), dim3((unsigned)cells, s.tiles),
                           dim3(64 * s.team), 0, stream, p, s, s.bc);
        e = hipGetLastError();
    }
    if (e != hipSuccess)
        return e;
    if (!p.out) {
        hipLaunchKernelGGL(ssu_scan_last_kernel, dim3((unsigned)(p.batch * s.blocks), s.tiles),
                           dim3(1024), 0, stream, p, s);
        return hipGetLastError();
    }
    const int lds = 4 * 64 * s.team * s.tiles *
                    ((s.chunks > 1 ? kStates : 0) + (s.tiles > 1 ? 2 * kBatch : 0));
    if (s.tiles == 1) {
        hipLaunchKernelGGL((ssu_scan_tokens_kernel<IOT, DTT, true>), dim3((unsigned)cells),
                           dim3(64 * s.team), lds, stream, p, s, s.bc, p.out);
        return hipGetLastError();
    }
    static std::atomic<uint64_t> raised{0};
    e = raise_lds(reinterpret_cast<const void *>(ssu_scan_tokens_kernel<IOT, DTT, false>), lds, &raised);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((ssu_scan_tokens_kernel<IOT, DTT, false>), dim3((unsigned)cells),
                       dim3(64 * s.tiles * s.team), lds, stream, p, s, s.bc, p.out);
    return hipGetLastError();
}

template <typename IOT, typename DTT, int BC>
hipError_t launch_sweep(const ScanParams &p, hipStream_t stream)
{
    const int per_group = (p.dim / p.ngroups + 15) / 16, blocks = per_group * p.ngroups;
    const int tiles = (p.dstate + kStates - 1) / kStates;
    if ((int64_t)p.batch * blocks > 0x7fffffff)
        return hipErrorInvalidConfiguration;
    const int lds = 4 * (kSweepWaves * 16 * kVuPitch + 2 * kSweepWaves * 64 * 8 + 2 * tiles * 64 * 4);
    const auto kernel = ssu_scan_sweep_kernel<IOT, DTT, BC>;
    static std::atomic<uint64_t> raised{0};
    const hipError_t e = raise_lds(reinterpret_cast<const void *>(kernel), lds, &raised);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(p.batch * blocks)), dim3(64 * kSweepWaves), lds, stream,
                       p, per_group, blocks, tiles);
    return hipGetLastError();
}

template <typename IOT, typename DTT>
hipError_t launch_prompt(const ScanParams &p, const Plan &q, hipStream_t stream)
{
    if (!q.sweep)
        return launch_chunks<IOT, DTT>(p, q, stream);
    const int es = p.bc_dtype == kF32 ? 4 : 2;
    auto vec = [&](const void *m, int64_t bs, int64_t ts) {
        return (uintptr_t)m % (4 * es) == 0 && bs % 4 == 0 && ts % 4 == 0;
    };
    if (!vec(p.B, p.b_bs, p.b_ts) || (p.out && !vec(p.C, p.c_bs, p.c_ts)))
        return launch_sweep<IOT, DTT, 0>(p, stream);
    return es == 4 ? launch_sweep<IOT, DTT, 4>(p, stream) : launch_sweep<IOT, DTT, 2>(p, stream);
}

template <typename IOT>
hipError_t launch_prompt_dt(const ScanParams &p, const Plan &q, hipStream_t stream)
{
    switch (p.dt_dtype) {
    case kF32: return launch_prompt<IOT, float>(p, q, stream);
    case kF16: return launch_prompt<IOT, _Float16>(p, q, stream);
    default: return launch_prompt<IOT, bf16_t>(p, q, stream);
    }
}

}  // namespace

int64_t scan_workspace_floats(int64_t batch, int64_t dim, int64_t dstate, int64_t ngroups,
                              int64_t seq_len)
{
    const Plan q = scan_plan(batch, dim, dstate, ngroups, seq_len, true);  // the finer cut
    return q.bc_floats + q.start_floats + q.sum_floats;
}

hipError_t launch_scan(const ScanParams &p, hipStream_t stream)
{
    (void)hipGetLastError();  // report only this launch's status
    Plan q = scan_plan(p.batch, p.dim, p.dstate, p.ngroups, p.seq_len, p.ctx != nullptr);
    if (!q.rows) {
        q.s.bc = p.workspace;
        q.s.zeros = q.bc_floats - 2 * kStates;
        q.s.start = q.s.bc + q.bc_floats;
        q.s.sum = q.s.start + q.start_floats;
        switch (p.io_dtype) {
        case kF32: return launch_prompt_dt<float>(p, q, stream);
        case kF16: return launch_prompt_dt<_Float16>(p, q, stream);
        default: return launch_prompt_dt<bf16_t>(p, q, stream);
        }
    }
    switch (p.state_dtype) {
    case kF32: return launch_rows_lanes<float>(p, stream);
    case kF16: return launch_rows_lanes<_Float16>(p, stream);
    default: return launch_rows_lanes<bf16_t>(p, stream);
    }
}

}  // namespace ssu
