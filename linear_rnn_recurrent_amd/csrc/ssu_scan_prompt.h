// Per-channel selective scan of prompts: the kernels of ssu_scan.hip's other two
// evaluations, which that file describes. Instantiated once per type of x, z and
// out by ssu_scan_prompt_{f32,f16,bf16}.hip.
#pragma once

#include <algorithm>

#include "ssu_scan_impl.h"

namespace ssu {
namespace {

// ---------------------------------------------------------------------------
// Chunks
// ---------------------------------------------------------------------------
// The block of channels, the batch row and the team of chunks of a workgroup.
struct Place {
    int b, team, blk, g, d, dl;  // .., group, channel (clamped), whether its lane is live
};

__device__ __forceinline__ Place place(const ScanParams &p, const ChunkShape &s, int teams, int first = 0)
{
    Place q;
    int i = first + blockIdx.x;
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
        a[j] = log2_rate(w.x);
        a[j + 1] = log2_rate(w.y);
        a[j + 2] = log2_rate(w.z);
        a[j + 3] = log2_rate(w.w);
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

// The pool's entries of a lane (0 past dstate), all on their way at once.
__device__ __forceinline__ void load_states(const ScanParams &p, int64_t so, int tile, float (&h)[kStates])
{
    auto load = [&](auto f32) {
        constexpr int SZ = decltype(f32)::value ? 4 : 2;
        Raw4x w[kStates / 4];
#pragma unroll
        for (int j = 0; j < kStates; j += 4)
            w[j / 4] = raw4<SZ>(p.state, so + (tile * kStates + j < p.dstate ? j : 0), p.state_dtype);
#pragma unroll
        for (int j = 0; j < kStates; j += 4) {
            float v[4];
            cvt4<SZ>(w[j / 4], p.state_dtype, v);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                h[j + k] = tile * kStates + j < p.dstate ? v[k] : 0.0f;
        }
    };
    if (p.state_dtype == kF32)
        load(std::true_type());
    else
        load(std::false_type());
}

// Waits for v, values of scalar loads. Those return in any order, so that any
// wait is for all of them: loads are issued after the wait for the ones before.
__device__ __forceinline__ void arrived(const float (&v)[kStates])
{
    asm volatile("" ::"s"(v[0]), "s"(v[1]), "s"(v[2]), "s"(v[3]), "s"(v[4]), "s"(v[5]), "s"(v[6]),
                 "s"(v[7]), "s"(v[8]), "s"(v[9]), "s"(v[10]), "s"(v[11]), "s"(v[12]), "s"(v[13]),
                 "s"(v[14]), "s"(v[15]));
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
        float h[kStates];
        load_states(p, so, tile, h);
#pragma unroll
        for (int j = 0; j < kStates; ++j)
            e[j * 64] = h[j];
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
            arrived(bs);
            __builtin_amdgcn_sched_barrier(0);
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
        a[j] = n < p.dstate ? log2_rate(p.A[(int64_t)q.d * p.dstate + n]) : 0.0f;
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
                    h[j] = fmaf(h[j], whole_decay(a[j], total[i]), end[i][j]);
            }
        }
    }
    use(to, h);
}

// The last state where no outputs are wanted; a wave has one state entry of a
// tile. `first`: the launch's first block.
__global__ __launch_bounds__(1024) void ssu_scan_last_kernel(const ScanParams p, const ChunkShape s,
                                                             int first)
{
    const Place q = place(p, s, 1, first);
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
        load_states(p, so, tile, h);
    }
    if (ONE && !live)
        return;
    // the batches of the team's first chunk, the longest (every wave meets the
    // barriers)
    const int batches = (min(s.chunk, len - (ONE ? t0 : c0 * s.chunk)) + kBatch - 1) / kBatch;
    float *part = lds + (s.chunks > 1 ? s.team * s.tiles * kStates * 64 : 0);
    if (!live)
        bc = s.zeros;
    float bs[kStates], cs[kStates];  // the next token's B and C
#pragma unroll
    for (int j = 0; j < kStates; ++j)
        bs[j] = packed[bc + j], cs[j] = packed[bc + kStates + j];
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
        // token i + 1's B and C are on their way while token i is computed
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            bc = t + i + 1 < t1 ? bc + bc_step : s.zeros;
            arrived(bs);
            arrived(cs);
            __builtin_amdgcn_sched_barrier(0);
            float bn[kStates], cn[kStates];
#pragma unroll
            for (int j = 0; j < kStates; ++j)
                bn[j] = packed[bc + j], cn[j] = packed[bc + kStates + j];
            float y2[2] = {0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < kStates; ++j) {
                h[j] = fmaf(h[j], __builtin_amdgcn_exp2f(a[j] * v[i]), u[i] * bs[j]);
                y2[j & 1] = fmaf(h[j], cs[j], y2[j & 1]);
                bs[j] = bn[j];
                cs[j] = cn[j];
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
constexpr int vu_pitch(int sub) { return 2 * sub + 4; }  // floats: the channels on different banks

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

// The row with the n-th most tokens (at most 64 rows; ties in order).
__device__ __forceinline__ int nth_longest(const ScanParams &p, int n)
{
    const int i = threadIdx.x & 63;
    int row, mine = -1, rank = 0;
    if (i < p.batch)
        mine = row_tokens(p, i, &row);
    for (int j = 0; j < p.batch; ++j) {
        const int other = __builtin_amdgcn_readlane(mine, j);
        rank += other > mine || (other == mine && j < i);
    }
    return __ffsll((unsigned long long)__ballot(i < p.batch && rank == n)) - 1;
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

// A workgroup of WAVES waves sweeps 16 channels through a row's tokens, kSub
// tokens a wave and step. Lane (r, c) of a wave has four state entries (4r ..) of
// channel c: it runs the wave's tokens from a zero start keeping the kSub decays of
// each entry, the waves exchange ends and decays through LDS, and every wave runs
// its tokens again from its true start without any exponential. A token's B lies
// across the 16 lanes of a row and reaches its channels by the DPP of a product; C,
// whose multiply-adds do not take one here, goes through the wave's own LDS (by DPP
// as well: 52 us for 49 at 4 x 512 x 2560), and so do dt' and dt' x, two tokens a
// read (one: 49 us for 46). The sum over dstate is two swap-and-adds that also hand
// lane (r, c) the outputs of kSub / 4 tokens, those whose x, dt and z it loaded.
// dstate above 16 repeats the two runs per 16.
//
// kSub: 16 spreads a step's exchange over more tokens, 8 wastes less at the rows'
// ends and holds half the decays. 4 waves are what short and uneven rows take, with
// 8 (us with 8 | 16: 8 x 777 x 2560 uneven 74 | 77, 32 x 128 x 2560 73 | 80,
// 4 x 512 x 2560 51 | 47, where 8 waves take 45); 8 and 16 waves take longer rows,
// with 16 (8 waves, with 8 | 16: 4 x 512 x 2560 50 | 45, 1 x 2048 x 1536 88 | 74; 16
// waves: 1 x 2048 x 1536 71 | 60, 2 x 509 x 1536 dstate 64 59 | 51). The rest beside
// the vector ALU is the exchange's barriers and the rows' ends. Four waves a SIMD
// leave the 128 registers that kSub 16 needs: at five it spills (115 us for 64, before
// C went through LDS).
template <typename IOT, typename DTT, int BC, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 4) void ssu_scan_sweep_kernel(
    const ScanParams p, int per_group, int blocks, int tiles)
{
    extern __shared__ float lds[];
    constexpr int kSub = sweep_tokens(WAVES);
    constexpr int kOwn = kSub / 4, kVuPitch = vu_pitch(kSub);  // a lane loads and finishes kOwn tokens
    // [waves][16][kVuPitch] dt', dt' x; [2][waves][64][8] ends and decays; [2][tiles][64][4] states;
    // [waves][kSub][4][4] C
    const int lane = threadIdx.x & 63, r = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float *vu = lds + wave * (16 * kVuPitch);
    float4 *ends = reinterpret_cast<float4 *>(lds + WAVES * 16 * kVuPitch);
    float4 *starts = ends + 2 * WAVES * 64 * 2;
    float4 *cl = starts + 2 * tiles * 64 + wave * (kSub * 4);  // [token][r] C

    // eight neighbouring blocks, which share cache lines of x, dt, z and out, on
    // one XCD (workgroups go to the eight XCDs in turn)
    int id = blockIdx.x;
    if (id < (int)(gridDim.x & ~63u))
        id = (id & ~63) + (id & 7) * 8 + ((id >> 3) & 7);
    const int turn = id / blocks, blk = id - turn * blocks;
    // rows of uneven lengths start longest first
    const int b = p.ctx && p.batch <= 64 ? nth_longest(p, turn) : turn;
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
        for (int t = len + wave * 4 + r; t < p.seq_len; t += WAVES * 4)
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
    for (int k = wave; k < tiles; k += WAVES) {
        float h[4] = {};
        const int n0 = k * kStates + r * 4;
        if (n0 < p.dstate)
            ld_state4(p, so + n0, h);
        starts[k * 64 + lane] = make_float4(h[0], h[1], h[2], h[3]);
    }
    int starts_now = 0;  // which of the two copies the step reads; the other gets the next's

    // a lane's byte offsets of its tokens from the wave's first (host: 16
    // token strides < 2^32 bytes)
    const uint32_t xts = (uint32_t)p.x_ts * SZ, gts = (uint32_t)zts * SZ, dts = (uint32_t)p.dt_ts * DZ,
                   ots = (uint32_t)p.out_ts * SZ;
    E x[kOwn], z[kOwn];
    DE dt[kOwn];
    auto load = [&](int t0) {  // this wave's tokens of the step at t0; past the row: its last
        const int w0 = min(t0 + wave * kSub, len - 1), most = len - 1 - w0;
        const char *xw = xp + w0 * p.x_ts * SZ, *zw = zp + w0 * zts * SZ, *dw = dp + w0 * p.dt_ts * DZ;
#pragma unroll
        for (int q = 0; q < kOwn; ++q) {
            const uint32_t t = min(r * kOwn + q, most);
            x[q] = *reinterpret_cast<const E *>(xw + (t * xts + dx));
            z[q] = *reinterpret_cast<const E *>(zw + (t * gts + dx));
            dt[q] = *reinterpret_cast<const DE *>(dw + (t * dts + dd));
        }
    };
    load(0);
    int buf = 0;
    for (int t0 = 0; t0 < len; t0 += kSub * WAVES) {
        const int w0 = t0 + wave * kSub;  // the wave's first token
        float xs[kOwn], gate[kOwn], y4[kOwn] = {};
#pragma unroll
        for (int q = 0; q < kOwn; ++q) {
            float v = cvt_raw1<DTT>(dt[q]) + bias;
            if (p.dt_softplus)
                v = softplus_f32(v);
            const bool in = w0 + r * kOwn + q < len;  // others are neutral: dt' = 0
            v = in ? v : 0.0f;
            const float xv = cvt_raw1<IOT>(x[q]);
            *reinterpret_cast<float2 *>(vu + c * kVuPitch + (r * kOwn + q) * 2) =
                make_float2(v, in ? v * xv : 0.0f);
            xs[q] = skip * xv;
            gate[q] = cvt_raw1<IOT>(z[q]);
        }
        __builtin_amdgcn_wave_barrier();
        if (t0 + kSub * WAVES < len)
            load(t0 + kSub * WAVES);
        for (int k = 0; k < tiles; ++k) {
            const int n0 = k * kStates + r * 4, nn = min(n0, p.dstate - 4);
            const bool own = n0 < p.dstate;
            const float4 aw = *reinterpret_cast<const float4 *>(p.A + (int64_t)d * p.dstate + nn);
            const int tok = min(w0 + c % kSub, len - 1);  // B and C: lane c has token c of the wave's
            float bv[4], cv[4];
            ld_bc4<BC>(bp + tok * bts, nn * bz, p.bc_dtype, bv);
            ld_bc4<BC>(cp + tok * cts, nn * bz, p.bc_dtype, cv);
            const float a[4] = {log2_rate(aw.x), log2_rate(aw.y), log2_rate(aw.z), log2_rate(aw.w)};
            const bool real = own && w0 + c % kSub < len;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bv[j] = real ? bv[j] : 0.0f;
                cv[j] = real ? cv[j] : 0.0f;
            }
            cl[(c % kSub) * 4 + r] = make_float4(cv[0], cv[1], cv[2], cv[3]);
            // from a zero start
            float dec[kSub][4], h[4] = {}, sum = 0.0f;
            each_of(
                [&](auto tt) {
                    constexpr int t = decltype(tt)::value * 2;
                    const float4 w = *reinterpret_cast<const float4 *>(vu + c * kVuPitch + t * 2);
                    sum += w.x + w.z;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        dec[t][j] = __builtin_amdgcn_exp2f(a[j] * w.x);
                        dec[t + 1][j] = __builtin_amdgcn_exp2f(a[j] * w.z);
                        h[j] = fmaf(h[j], dec[t][j], row_lane<t>(bv[j]) * w.y);
                        h[j] = fmaf(h[j], dec[t + 1][j], row_lane<t + 1>(bv[j]) * w.w);
                    }
                    __builtin_amdgcn_sched_barrier(0);  // keeps the tokens in order, and the registers few
                },
                std::make_integer_sequence<int, kSub / 2>());
            float4 *mine = ends + ((buf * WAVES + wave) * 64 + lane) * 2;
            mine[0] = make_float4(h[0], h[1], h[2], h[3]);
            mine[1] = make_float4(whole_decay(a[0], sum), whole_decay(a[1], sum), whole_decay(a[2], sum),
                                  whole_decay(a[3], sum));
            __syncthreads();
            // the wave's start
            const float4 s0 = starts[(starts_now * tiles + k) * 64 + lane];
            h[0] = s0.x, h[1] = s0.y, h[2] = s0.z, h[3] = s0.w;
            for (int m = 0; m < wave; ++m) {
                const float4 e = ends[((buf * WAVES + m) * 64 + lane) * 2];
                const float4 f = ends[((buf * WAVES + m) * 64 + lane) * 2 + 1];
                h[0] = fmaf(h[0], f.x, e.x);
                h[1] = fmaf(h[1], f.y, e.y);
                h[2] = fmaf(h[2], f.z, e.z);
                h[3] = fmaf(h[3], f.w, e.w);
            }
            buf ^= 1;
            float y[kSub];
            each_of(
                [&](auto tt) {
                    constexpr int t = decltype(tt)::value * 2;
                    const float4 w = *reinterpret_cast<const float4 *>(vu + c * kVuPitch + t * 2);
                    const float4 c0 = cl[t * 4 + r], c1 = cl[t * 4 + 4 + r];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        h[j] = fmaf(h[j], dec[t][j], row_lane<t>(bv[j]) * w.y);
                    y[t] = fmaf(h[3], c0.w, fmaf(h[2], c0.z, fmaf(h[1], c0.y, h[0] * c0.x)));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        h[j] = fmaf(h[j], dec[t + 1][j], row_lane<t + 1>(bv[j]) * w.w);
                    y[t + 1] = fmaf(h[3], c1.w, fmaf(h[2], c1.z, fmaf(h[1], c1.y, h[0] * c1.x)));
                    __builtin_amdgcn_sched_barrier(0);
                },
                std::make_integer_sequence<int, kSub / 2>());
            // sums over the four rows: halves, then rows, leaving the lane's own tokens
            float y8[2 * kOwn];
#pragma unroll
            for (int i = 0; i < 2 * kOwn; ++i) {
                const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(y[i]),
                                                                __float_as_uint(y[i + 2 * kOwn]), false, false);
                y8[i] = __uint_as_float(w[0]) + __uint_as_float(w[1]);
            }
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(y8[i]),
                                                                __float_as_uint(y8[i + kOwn]), false, false);
                y4[i] += __uint_as_float(w[0]) + __uint_as_float(w[1]);
            }
            if (wave == WAVES - 1)
                starts[((starts_now ^ 1) * tiles + k) * 64 + lane] = make_float4(h[0], h[1], h[2], h[3]);
        }
        if (p.out) {
#pragma unroll
            for (int q = 0; q < kOwn; ++q) {
                float v = y4[q] + xs[q];
                if (gated)
                    v *= silu_hw(gate[q]);
                if (w0 + r * kOwn + q < len)
                    put<IOT>(out + w0 * p.out_ts * SZ + ((r * kOwn + q) * ots + dx), v);
            }
        }
        starts_now ^= 1;
    }
    __syncthreads();
    if (p.update) {
        for (int k = wave; k < tiles; k += WAVES) {
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

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
// Dynamic LDS above the default 64 KiB (up to a CU's 160) is allowed once per
// kernel and device.
hipError_t raise_lds(const void *kernel, int bytes, std::atomic<uint64_t> *raised)
{
    if (bytes <= 65536)
        return hipSuccess;
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess || (dev < 64 && ((raised->load(std::memory_order_relaxed) >> dev) & 1)))
        return e;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 163840);
    if (e == hipSuccess && dev < 64)
        raised->fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

template <typename IOT, typename DTT>
hipError_t launch_chunks(const ScanParams &p, const ScanPlan &q, hipStream_t stream)
{
    const ChunkShape &s = q.s;
    const int64_t cells = (int64_t)p.batch * s.blocks * ((s.chunks + s.team - 1) / s.team);
    const int64_t packed = q.bc_floats / 2 - kStates;
    if (!launchable(cells, 64 * s.team * s.tiles) || !launchable((packed + 255) / 256, 256))
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
        constexpr int MOST = 1 << 21;  // workgroups of a launch: 2^31 threads
        for (int first = 0; e == hipSuccess && first < p.batch * s.blocks; first += MOST) {
            hipLaunchKernelGGL(ssu_scan_last_kernel,
                               dim3((unsigned)std::min(MOST, p.batch * s.blocks - first), s.tiles),
                               dim3(1024), 0, stream, p, s, first);
            e = hipGetLastError();
        }
        return e;
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

template <typename IOT, typename DTT, int BC, int WAVES>
hipError_t launch_sweep(const ScanParams &p, hipStream_t stream)
{
    const int per_group = (p.dim / p.ngroups + 15) / 16, blocks = per_group * p.ngroups;
    const int tiles = (p.dstate + kStates - 1) / kStates;
    if (!launchable((int64_t)p.batch * blocks, 64 * WAVES))
        return hipErrorInvalidConfiguration;
    const int lds = 4 * (WAVES * 16 * vu_pitch(sweep_tokens(WAVES)) + 2 * WAVES * 64 * 8 + 2 * tiles * 64 * 4 +
                         WAVES * sweep_tokens(WAVES) * 16);
    const auto kernel = ssu_scan_sweep_kernel<IOT, DTT, BC, WAVES>;
    static std::atomic<uint64_t> raised{0};
    const hipError_t e = raise_lds(reinterpret_cast<const void *>(kernel), lds, &raised);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(p.batch * blocks)), dim3(64 * WAVES), lds, stream,
                       p, per_group, blocks, tiles);
    return hipGetLastError();
}

template <typename IOT, typename DTT, int BC>
hipError_t launch_sweep_waves(const ScanParams &p, const ScanPlan &q, hipStream_t stream)
{
    switch (q.sweep) {
    case 4: return launch_sweep<IOT, DTT, BC, 4>(p, stream);
    case 8: return launch_sweep<IOT, DTT, BC, 8>(p, stream);
    default: return launch_sweep<IOT, DTT, BC, 16>(p, stream);
    }
}

template <typename IOT, typename DTT>
hipError_t launch_prompt(const ScanParams &p, const ScanPlan &q, hipStream_t stream)
{
    if (!q.sweep)
        return launch_chunks<IOT, DTT>(p, q, stream);
    const int es = p.bc_dtype == kF32 ? 4 : 2;
    auto vec = [&](const void *m, int64_t bs, int64_t ts) {
        return (uintptr_t)m % (4 * es) == 0 && bs % 4 == 0 && ts % 4 == 0;
    };
    if (!vec(p.B, p.b_bs, p.b_ts) || (p.out && !vec(p.C, p.c_bs, p.c_ts)))
        return launch_sweep_waves<IOT, DTT, 0>(p, q, stream);
    return es == 4 ? launch_sweep_waves<IOT, DTT, 4>(p, q, stream)
                   : launch_sweep_waves<IOT, DTT, 2>(p, q, stream);
}

template <typename IOT>
hipError_t launch_prompt_dt(const ScanParams &p, const ScanPlan &q, hipStream_t stream)
{
    switch (p.dt_dtype) {
    case kF32: return launch_prompt<IOT, float>(p, q, stream);
    case kF16: return launch_prompt<IOT, _Float16>(p, q, stream);
    default: return launch_prompt<IOT, bf16_t>(p, q, stream);
    }
}

}  // namespace
}  // namespace ssu
