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
//   carry   every chunk's start from the ends before it, in order
//   tokens  every chunk's tokens from its start: the outputs, the last state
// (a single chunk is pack and tokens; without outputs the carry leaves the
// last state and the tokens are not run)
// The chunks' decays are computed twice (11 slots instead of 6), against 1/16
// of the SIMDs busy without the cut at one sequence of 5,120 channels. dstate
// above 16 takes ceil(dstate / 16) waves, whose partial outputs meet in LDS.
#include "ssu_device.h"
#include "ssu_dpp.h"
#include "ssu_internal.h"

namespace ssu {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kStates = 16;  // state entries of a lane in the chunk kernels
constexpr int kBatch = 8;    // tokens loaded together

// Elements by size: 4 bytes fp32, 2 bytes bf16 or fp16 (a uniform choice).
template <int SZ>
__device__ __forceinline__ uint32_t ld_bits(const void *p, int64_t i)
{
    if constexpr (SZ == 4)
        return static_cast<const uint32_t *>(p)[i];
    else
        return static_cast<const uint16_t *>(p)[i];
}
template <int SZ>
__device__ __forceinline__ float cvt_bits(uint32_t w, bool bf)
{
    if constexpr (SZ == 4)
        return __uint_as_float(w);
    else
        return bf ? __uint_as_float(w << 16) : f16_to_f32(w);
}
template <int SZ>
__device__ __forceinline__ void st_bits(void *p, int64_t i, float v, bool bf)
{
    if constexpr (SZ == 4)
        static_cast<float *>(p)[i] = v;
    else
        static_cast<uint16_t *>(p)[i] = (uint16_t)(bf ? f32_to_bf16(v) : f32_to_f16(v));
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
template <int LPC>
__global__ __launch_bounds__(256) void ssu_scan_rows_kernel(const ScanParams p)
{
    constexpr int CH = 256 / LPC;  // channels per workgroup
    const int sub = threadIdx.x & (LPC - 1);
    const int ch = threadIdx.x / LPC;
    const int tiles = (p.dim + CH - 1) / CH;
    const int b = blockIdx.x / tiles;
    const int d_raw = (blockIdx.x - b * tiles) * CH + ch;
    const int d = min(d_raw, p.dim - 1);
    const int n0 = sub * 4;
    const bool own = n0 < p.dstate;
    const bool writes = own && d_raw < p.dim;
    const bool head = sub == 0 && d_raw < p.dim;
    int row;
    const int len = row_tokens(p, b, &row);
    const int g = d / (p.dim / p.ngroups);
    const int64_t so = (int64_t)row * p.row_stride + (int64_t)d * p.dstate + n0;

    float h[4] = {}, a[4] = {};
    if (own && len > 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = p.A[(int64_t)d * p.dstate + n0 + j];
            h[j] = ld_io(p.state, so + j, p.state_dtype);
        }
    }
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.0f;
    const float skip = p.D ? p.D[d] : 0.0f;
    for (int t = 0; t < len; ++t) {
        float v = ld_io(p.dt, b * p.dt_bs + t * p.dt_ts + d, p.dt_dtype) + bias;
        if (p.dt_softplus)
            v = softplus_f32(v);
        const float x = ld_io(p.x, b * p.x_bs + t * p.x_ts + d, p.io_dtype);
        const int64_t bo = b * p.b_bs + t * p.b_ts + (int64_t)g * p.dstate + n0;
        const int64_t co = b * p.c_bs + t * p.c_ts + (int64_t)g * p.dstate + n0;
        const float u = v * x;
        float y = 0.0f;
        if (own) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = fmaf(u, ld_io(p.B, bo + j, p.bc_dtype), h[j] * expf(a[j] * v));
                if (p.out)
                    y = fmaf(h[j], ld_io(p.C, co + j, p.bc_dtype), y);
            }
        }
        if (p.out) {
            y = group_sum<LPC>(y);
            if (head) {
                y = fmaf(skip, x, y);
                if (p.z)
                    y *= silu_f32(ld_io(p.z, b * p.z_bs + t * p.z_ts + d, p.io_dtype));
                st_io(p.out, b * p.out_bs + t * p.out_ts + d, y, p.io_dtype);
            }
        }
    }
    if (p.out && head)
        for (int t = len; t < p.seq_len; ++t)
            st_io(p.out, b * p.out_bs + t * p.out_ts + d, 0.0f, p.io_dtype);
    if (p.update && writes && len > 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            st_io(p.state, so + j, h[j], p.state_dtype);
    }
}

template <int LPC>
hipError_t launch_scan_lanes(const ScanParams &p, hipStream_t stream)
{
    const int64_t blocks = (int64_t)p.batch * ((p.dim + 256 / LPC - 1) / (256 / LPC));
    if (blocks > 0x7fffffff)
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(ssu_scan_rows_kernel<LPC>, dim3((unsigned)blocks), dim3(256), 0, stream, p);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Chunks
// ---------------------------------------------------------------------------
// Workspace, in floats: packed B | C [batch][seq_len][ngroups][tiles][2][16],
// chunk starts [batch][chunks][blocks][tiles][16][64] (slot c + 1 holds chunk
// c's end until the carry kernel replaces it by chunk c + 1's start), chunk
// sums of dt' [batch][chunks][blocks][64]. A block is 64 channels of one group.
struct ChunkShape {
    int32_t tiles, per_group, blocks, chunk, chunks;
    float *bc, *start, *sum;
};

// The block of channels and the chunk of a workgroup.
struct Place {
    int b, c, blk, g, d, dl;  // batch row, chunk, block, group, channel (clamped), its lane is live
};

__device__ __forceinline__ Place place(const ScanParams &p, const ChunkShape &s, int chunks)
{
    Place q;
    int i = blockIdx.x;
    q.blk = i % s.blocks;
    i /= s.blocks;
    q.c = i % chunks;
    q.b = i / chunks;
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

// A batch of tokens' inputs as raw bits.
template <int IOSZ, int DTSZ>
struct Inputs {
    uint32_t x[kBatch], dt[kBatch];
    __device__ __forceinline__ void load(const ScanParams &p, const Place &q, int t0, int t1)
    {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int t = min(t0 + i, t1 - 1);
            x[i] = ld_bits<IOSZ>(p.x, q.b * p.x_bs + t * p.x_ts + q.d);
            dt[i] = ld_bits<DTSZ>(p.dt, q.b * p.dt_bs + t * p.dt_ts + q.d);
        }
    }
};

template <int DTSZ>
__device__ __forceinline__ float step_size(uint32_t bits, float bias, const ScanParams &p, bool bf)
{
    const float v = cvt_bits<DTSZ>(bits, bf) + bias;
    return p.dt_softplus ? softplus_f32(v) : v;
}

// Every chunk's end from a zero start (all but a row's last chunk, or all of
// them where only the state is wanted).
template <int IOSZ, int DTSZ>
__global__ __launch_bounds__(64, 4) void ssu_scan_ends_kernel(const ScanParams p, const ChunkShape s,
                                                              const float *__restrict__ packed)
{
    const Place q = place(p, s, s.chunks);
    const int tile = blockIdx.y;
    int row;
    const int len = row_tokens(p, q.b, &row);
    const int t0 = q.c * s.chunk, t1 = min(t0 + s.chunk, len);
    if (t0 >= len || (p.out && t1 == len))
        return;
    const float *bc = packed + ((((int64_t)q.b * p.seq_len + t0) * p.ngroups + q.g) * s.tiles + tile) *
                                 (2 * kStates);
    const int64_t bc_step = (int64_t)p.ngroups * s.tiles * 2 * kStates;
    const bool io_bf = p.io_dtype == kBF16, dt_bf = p.dt_dtype == kBF16;
    const float bias = p.dt_bias ? p.dt_bias[q.d] : 0.0f;
    float a[kStates], h[kStates] = {}, sum = 0.0f;
    load_a(p, q.d, tile, a);
    Inputs<IOSZ, DTSZ> in;
    in.load(p, q, t0, t1);
    for (int t = t0; t < t1; t += kBatch) {
        const Inputs<IOSZ, DTSZ> now = in;
        if (t + kBatch < t1)
            in.load(p, q, t + kBatch, t1);
        auto token = [&](int i) {
            const float v = step_size<DTSZ>(now.dt[i], bias, p, dt_bf);
            const float u = v * cvt_bits<IOSZ>(now.x[i], io_bf);
            sum += v;
#pragma unroll
            for (int j = 0; j < kStates; ++j)
                h[j] = fmaf(h[j], __builtin_amdgcn_exp2f(a[j] * v), u * bc[i * bc_step + j]);
        };
        if (t + kBatch <= t1) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                token(i);
        } else {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (t + i < t1)
                    token(i);
        }
        bc += kBatch * bc_step;
    }
    const int lane = threadIdx.x;
    const int64_t at = ((int64_t)q.b * (s.chunks + 1) + q.c + 1) * s.blocks + q.blk;
    float *e = s.start + (at * s.tiles + tile) * (kStates * 64) + lane;
#pragma unroll
    for (int j = 0; j < kStates; ++j)
        e[j * 64] = h[j];
    if (tile == 0)
        s.sum[at * 64 + lane] = sum;
}

// Every chunk's start, from the pool's state and the ends in order; with no
// outputs also the row's last state. A wave has four state entries of a tile.
__global__ __launch_bounds__(256) void ssu_scan_carry_kernel(const ScanParams p, const ChunkShape s)
{
    const Place q = place(p, s, 1);
    const int tile = blockIdx.y;
    int row;
    const int len = row_tokens(p, q.b, &row);
    if (len == 0)
        return;
    const int lane = threadIdx.x & 63;
    const int j0 = (threadIdx.x >> 6) * 4, n0 = tile * kStates + j0;
    const bool own = n0 < p.dstate;
    const int64_t so = (int64_t)row * p.row_stride + (int64_t)q.d * p.dstate + n0;
    float a[4] = {}, h[4] = {};
    if (own) {
        const float4 w = *reinterpret_cast<const float4 *>(p.A + (int64_t)q.d * p.dstate + n0);
        a[0] = w.x * kLog2e, a[1] = w.y * kLog2e, a[2] = w.z * kLog2e, a[3] = w.w * kLog2e;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            h[j] = ld_io(p.state, so + j, p.state_dtype);
    }
    const int n = (len + s.chunk - 1) / s.chunk;  // the row's chunks
    const int ends = p.out ? n - 1 : n;
    const int64_t step = (int64_t)s.blocks * s.tiles * (kStates * 64);
    float *e = s.start + ((((int64_t)q.b * (s.chunks + 1)) * s.blocks + q.blk) * s.tiles + tile) *
                             (kStates * 64) + j0 * 64 + lane;
    const float *sum = s.sum + (((int64_t)q.b * (s.chunks + 1)) * s.blocks + q.blk) * 64 + lane;
    if (p.out) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            e[j * 64] = h[j];
    }
    constexpr int F = 4;  // ends in flight
    for (int c = 0; c < ends; c += F) {
        float end[F][4], total[F];
#pragma unroll
        for (int i = 0; i < F; ++i) {
            const int k = min(c + i, ends - 1) + 1;
            total[i] = sum[(int64_t)k * s.blocks * 64];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                end[i][j] = e[k * step + j * 64];
        }
#pragma unroll
        for (int i = 0; i < F; ++i) {
            if (c + i < ends) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[j] = fmaf(h[j], __builtin_amdgcn_exp2f(a[j] * total[i]), end[i][j]);
                    if (p.out)
                        e[(c + i + 1) * step + j * 64] = h[j];
                }
            }
        }
    }
    if (!p.out && p.update && own && q.dl) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            st_io(p.state, so + j, h[j], p.state_dtype);
    }
}

// The tokens of every chunk from its start. tiles waves, one per 16 state
// entries; with more than one, a batch's partial outputs are summed through
// LDS (two buffers, so one barrier a batch) and its tokens finished by the
// waves in turn.
template <int IOSZ, int DTSZ, bool ONE>
__global__ __launch_bounds__(ONE ? 64 : 1024, 4) void ssu_scan_tokens_kernel(
    const ScanParams p, const ChunkShape s, const float *__restrict__ packed,
    void *__restrict__ out)
{
    extern __shared__ float part[];  // [2][tiles][kBatch][64] unless ONE
    const Place q = place(p, s, s.chunks);
    const int lane = threadIdx.x & 63;
    const int tile = ONE ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int row;
    const int len = row_tokens(p, q.b, &row);
    const int t0 = q.c * s.chunk, t_end = min(t0 + s.chunk, p.seq_len), t1 = min(t_end, len);
    const bool io_bf = p.io_dtype == kBF16, dt_bf = p.dt_dtype == kBF16;
    const int64_t oo = q.b * p.out_bs + q.d;
    if (out && q.dl)
        for (int t = max(t0, len) + tile; t < t_end; t += ONE ? 1 : s.tiles)
            st_bits<IOSZ>(out, oo + t * p.out_ts, 0.0f, io_bf);
    if (t0 >= len)
        return;

    const float *bc = packed + ((((int64_t)q.b * p.seq_len + t0) * p.ngroups + q.g) * s.tiles + tile) *
                                 (2 * kStates);
    const int64_t bc_step = (int64_t)p.ngroups * s.tiles * 2 * kStates;
    const float bias = p.dt_bias ? p.dt_bias[q.d] : 0.0f;
    const float skip = p.D ? p.D[q.d] : 0.0f;
    const int64_t so = (int64_t)row * p.row_stride + (int64_t)q.d * p.dstate + tile * kStates;
    float a[kStates], h[kStates] = {};
    load_a(p, q.d, tile, a);
    if (s.chunks > 1) {
        const int64_t at = ((int64_t)q.b * (s.chunks + 1) + q.c) * s.blocks + q.blk;
        const float *e = s.start + (at * s.tiles + tile) * (kStates * 64) + lane;
#pragma unroll
        for (int j = 0; j < kStates; ++j)
            h[j] = e[j * 64];
    } else {
#pragma unroll
        for (int j = 0; j < kStates; ++j)
            if (tile * kStates + (j & ~3) < p.dstate)
                h[j] = ld_io(p.state, so + j, p.state_dtype);
    }
    const void *zsrc = p.z ? p.z : p.x;  // without a gate: loaded and not used
    const int64_t zb = p.z ? p.z_bs : p.x_bs, zt = p.z ? p.z_ts : p.x_ts;
    Inputs<IOSZ, DTSZ> in;
    uint32_t zin[kBatch];
    auto load = [&](int t) {
        in.load(p, q, t, t1);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            zin[i] = ld_bits<IOSZ>(zsrc, q.b * zb + min(t + i, t1 - 1) * zt + q.d);
    };
    auto finish = [&](float y, float x, uint32_t zbits, int t) {
        y = fmaf(skip, x, y);
        if (p.z)
            y *= silu_hw(cvt_bits<IOSZ>(zbits, io_bf));
        if (out && q.dl)
            st_bits<IOSZ>(out, oo + t * p.out_ts, y, io_bf);
    };
    load(t0);
    int buf = 0;
    for (int t = t0; t < t1; t += kBatch) {
        const Inputs<IOSZ, DTSZ> now = in;
        uint32_t znow[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            znow[i] = zin[i];
        if (t + kBatch < t1)
            load(t + kBatch);
        auto token = [&](int i) {
            const float v = step_size<DTSZ>(now.dt[i], bias, p, dt_bf);
            const float x = cvt_bits<IOSZ>(now.x[i], io_bf);
            const float u = v * x;
            const float *w = bc + i * bc_step;
            float y[2] = {0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < kStates; ++j) {
                h[j] = fmaf(h[j], __builtin_amdgcn_exp2f(a[j] * v), u * w[j]);
                y[j & 1] = fmaf(h[j], w[kStates + j], y[j & 1]);
            }
            if constexpr (ONE)
                finish(y[0] + y[1], x, znow[i], t + i);
            else
                part[((buf * s.tiles + tile) * kBatch + i) * 64 + lane] = y[0] + y[1];
        };
        if (t + kBatch <= t1) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                token(i);
        } else {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (t + i < t1)
                    token(i);
        }
        if constexpr (!ONE) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (t + i < t1 && i % s.tiles == tile) {
                    float y = 0.0f;
                    for (int k = 0; k < s.tiles; ++k)
                        y += part[((buf * s.tiles + k) * kBatch + i) * 64 + lane];
                    finish(y, cvt_bits<IOSZ>(now.x[i], io_bf), znow[i], t + i);
                }
            }
            buf ^= 1;
        }
        bc += kBatch * bc_step;
    }
    if (p.update && t1 == len && q.dl) {
#pragma unroll
        for (int j = 0; j < kStates; ++j)
            if (tile * kStates + (j & ~3) < p.dstate)
                st_io(p.state, so + j, h[j], p.state_dtype);
    }
}

// Which evaluation a call takes, and its cut. The target is four waves on each
// SIMD of a full GPU (256 compute units, 4 SIMDs).
struct Plan {
    bool rows;
    ChunkShape s;
    int64_t bc_floats, start_floats, sum_floats;
};

Plan scan_plan(int64_t batch, int64_t dim, int64_t dstate, int64_t ngroups, int64_t seq_len)
{
    Plan q = {};
    q.rows = seq_len <= 16;
    if (q.rows)
        return q;
    q.s.tiles = (int32_t)((dstate + kStates - 1) / kStates);
    q.s.per_group = (int32_t)((dim / ngroups + 63) / 64);
    q.s.blocks = (int32_t)(q.s.per_group * ngroups);
    const int64_t waves = batch * q.s.blocks * q.s.tiles, target = 4096;
    int64_t chunks = waves >= target ? 1 : (target + waves - 1) / waves;
    int64_t len = (seq_len + chunks - 1) / chunks;
    len = (len + kBatch - 1) / kBatch * kBatch;
    if (len < 32)
        len = 32;
    chunks = (seq_len + len - 1) / len;
    q.s.chunk = (int32_t)(len > seq_len ? seq_len : len);
    q.s.chunks = (int32_t)chunks;
    q.bc_floats = batch * seq_len * ngroups * q.s.tiles * (2 * kStates);
    if (chunks > 1) {
        q.start_floats = batch * (chunks + 1) * q.s.blocks * q.s.tiles * (kStates * 64);
        q.sum_floats = batch * (chunks + 1) * q.s.blocks * 64;
    }
    return q;
}

template <int IOSZ, int DTSZ>
hipError_t launch_chunks(const ScanParams &p, const Plan &q, hipStream_t stream)
{
    const ChunkShape &s = q.s;
    const int64_t cells = (int64_t)p.batch * s.blocks * s.chunks;
    const int64_t packed = q.bc_floats / 2;
    if (cells > 0x7fffffff || (packed + 255) / 256 > 0x7fffffff)
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(ssu_scan_pack_kernel, dim3((unsigned)((packed + 255) / 256)), dim3(256), 0,
                       stream, p, s, packed);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && s.chunks > 1) {
        hipLaunchKernelGGL((ssu_scan_ends_kernel<IOSZ, DTSZ>), dim3((unsigned)cells, s.tiles),
                           dim3(64), 0, stream, p, s, s.bc);
        e = hipGetLastError();
        if (e == hipSuccess) {
            hipLaunchKernelGGL(ssu_scan_carry_kernel, dim3((unsigned)(p.batch * s.blocks), s.tiles),
                               dim3(256), 0, stream, p, s);
            e = hipGetLastError();
        }
    }
    if (e != hipSuccess || (s.chunks > 1 && !p.out))
        return e;
    if (s.tiles == 1)
        hipLaunchKernelGGL((ssu_scan_tokens_kernel<IOSZ, DTSZ, true>), dim3((unsigned)cells),
                           dim3(64), 0, stream, p, s, s.bc, p.out);
    else
        hipLaunchKernelGGL((ssu_scan_tokens_kernel<IOSZ, DTSZ, false>), dim3((unsigned)cells),
                           dim3(64 * s.tiles), 2 * s.tiles * kBatch * 64 * 4, stream, p, s, s.bc,
                           p.out);
    return hipGetLastError();
}

}  // namespace

int64_t scan_workspace_floats(int64_t batch, int64_t dim, int64_t dstate, int64_t ngroups,
                              int64_t seq_len)
{
    const Plan q = scan_plan(batch, dim, dstate, ngroups, seq_len);
    return q.bc_floats + q.start_floats + q.sum_floats;
}

hipError_t launch_scan(const ScanParams &p, hipStream_t stream)
{
    (void)hipGetLastError();  // report only this launch's status
    Plan q = scan_plan(p.batch, p.dim, p.dstate, p.ngroups, p.seq_len);
    if (!q.rows) {
        q.s.bc = p.workspace;
        q.s.start = q.s.bc + q.bc_floats;
        q.s.sum = q.s.start + q.start_floats;
        const bool io4 = p.io_dtype == kF32, dt4 = p.dt_dtype == kF32;
        if (io4)
            return dt4 ? launch_chunks<4, 4>(p, q, stream) : launch_chunks<4, 2>(p, q, stream);
        return dt4 ? launch_chunks<2, 4>(p, q, stream) : launch_chunks<2, 2>(p, q, stream);
    }
    if (p.dstate <= 4) return launch_scan_lanes<1>(p, stream);
    if (p.dstate <= 8) return launch_scan_lanes<2>(p, stream);
    if (p.dstate <= 16) return launch_scan_lanes<4>(p, stream);
    if (p.dstate <= 32) return launch_scan_lanes<8>(p, stream);
    if (p.dstate <= 64) return launch_scan_lanes<16>(p, stream);
    if (p.dstate <= 128) return launch_scan_lanes<32>(p, stream);
    return launch_scan_lanes<64>(p, stream);
}

}  // namespace ssu
