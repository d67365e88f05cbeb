// The gated delta rule token by token: single tokens, windows of drafted
// tokens, short prompts, and rows that are not 16-byte aligned.
//
//   S <- alpha S;  u = beta (v - S k);  S <- S + u k^T;  o = scale S q
//
// A value row of S (D keys) is independent of the others given k. KL lanes
// share a row, each with D / KL of its keys in runs of four (run j of lane l:
// keys 4 (l + KL j) .. + 3, so that one load instruction takes whole lines of
// the pool), and hold R adjacent rows. Both products of a token are taken with the
// state before it, o = scale (alpha S_old q + u (k . q)): they run side by
// side, and the chain from a token to the next is one product, its sum over KL
// lanes by DPP, and one multiply-add. The norms of q and k and their product
// are sums over the same lanes; the gates of 64 tokens are formed at once, one a lane.
// BLK tokens are read ahead, unconverted, so that a window waits for memory once.
//
// HBM bounds single tokens, by the state's read and write: 64 rows of 32 heads of 128 take
// 50.5 us, 270 MB at 5.35 TB/s. Windows: the state once, then the chain from token to token, 0.8 us
// a token (14 rows x 5, the state only read: 19.5 us, of which its 29 MB take 6).
#pragma once

#include "ssu_delta_impl.h"

namespace ssu {
namespace {

// lanes of a row, keys of a lane
template <int D>
struct DeltaLanes {
    static constexpr int KL = D >= 128 ? 16 : D / 8;
    static constexpr int KE = D / KL;
};

// N entries (a multiple of 2) of a row as their bits
template <typename IO, int N>
struct DeltaRun {
    uint32_t w[N * sizeof(IO) / 4];

    template <bool VEC>
    __device__ __forceinline__ void load(const IO *p)
    {
        constexpr int WORDS = N * sizeof(IO) / 4;
        if constexpr (VEC && WORDS == 4) {
            const u32x4 t = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = t[i];
        } else if constexpr (VEC && WORDS == 2) {
            const u32x2 t = *reinterpret_cast<const u32x2 *>(p);
            w[0] = t[0];
            w[1] = t[1];
        } else if constexpr (VEC && WORDS == 1) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                if constexpr (sizeof(IO) == 4)
                    w[e] = ld_raw1<IO>(p, e);
                else
                    w[e / 2] = e % 2 ? w[e / 2] | ld_raw1<IO>(p, e) << 16 : ld_raw1<IO>(p, e);
            }
        }
    }
    // From here on the values are used: without it the compiler moves conversions up to the loads
    __device__ __forceinline__ void arrive()
    {
#pragma unroll
        for (auto &x : w)
            asm volatile("" : "+v"(x));
    }
    __device__ __forceinline__ float operator[](int e) const
    {
        if constexpr (sizeof(IO) == 4)
            return __uint_as_float(w[e]);
        else if constexpr (__is_same(IO, bf16_t))
            return __uint_as_float(e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
        else
            return f16_to_f32(e % 2 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu);
    }
};

// Stores N (2 or 4) adjacent values
template <typename IO, int N, bool VEC>
__device__ __forceinline__ void delta_st_run(IO *p, const float (&v)[N])
{
    if constexpr (VEC && N == 4) {
        st_raw4<IO>(p, 0, v);
    } else if constexpr (VEC && sizeof(IO) == 2) {
        uint32_t h[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            h[k] = __is_same(IO, bf16_t) ? f32_to_bf16(v[k]) : f32_to_f16(v[k]);
        *reinterpret_cast<uint32_t *>(p) = h[0] | (h[1] << 16);
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
            st_elem<IO>(p, k, v[k]);
    }
}

// One wave: R G rows of value head h of batch entry b. BLK: tokens read ahead
// of their use (1: the call has one token).
template <typename IO, typename ST, int D, int R, int BLK, bool VEC>
__global__ __launch_bounds__(256) void delta_rows_kernel(DeltaParams p)
{
    constexpr int KL = DeltaLanes<D>::KL, KE = DeltaLanes<D>::KE;
    constexpr int N = KE / 4;       // runs of keys
    constexpr int G = 64 / KL;      // row groups of a wave
    constexpr int TILES = D / (G * R);  // waves a head
    static_assert(TILES * G * R == D, "rows of a head");
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t bh = wave / TILES;
    if (bh >= (int64_t)p.batch * p.hv)
        return;
    const int b = (int)(bh / p.hv), h = (int)(bh - (int64_t)b * p.hv);
    const int l = lane & (KL - 1), row0 = ((int)(wave - bh * TILES) * G + lane / KL) * R;
    const int pool = p.idx ? p.idx[b] : b;
    const int len = pool < 0 ? 0 : (p.ctx ? clamp_len(p.ctx[b], p.seq_len) : p.seq_len);
    const int jq = h / (p.hv / p.hq);
    const bool outs = p.out != nullptr;
    IO *op = static_cast<IO *>(p.out) + b * p.out_bs + (int64_t)h * D;

    if (len > 0) {
        ST *state = static_cast<ST *>(p.state) + pool * p.row_stride + (int64_t)h * D * D;
        const int s_off = row0 * D + 4 * l;
        typename Raw4<ST>::type w[R][N];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < N; ++j)
                w[r][j] = __builtin_nontemporal_load(reinterpret_cast<const typename Raw4<ST>::type *>(
                    state + s_off + r * D + 4 * KL * j));

        const IO *kp = static_cast<const IO *>(p.k) + b * p.k_bs + (int64_t)jq * D;
        // without outputs k is read in q's place
        const IO *qp = outs ? static_cast<const IO *>(p.q) + b * p.q_bs + (int64_t)jq * D : kp;
        const int64_t q_ts = outs ? p.q_ts : p.k_ts;
        const IO *vp = static_cast<const IO *>(p.v) + b * p.v_bs + (int64_t)h * D;
        DeltaRun<IO, 4> nk[BLK][N], nq[BLK][N];
        DeltaRun<IO, R> nv[BLK];
        auto load = [&](int t0) {  // tokens behind the end repeat the last one
#pragma unroll
            for (int i = 0; i < BLK; ++i) {
                const int64_t t = min(t0 + i, len - 1);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    nk[i][j].template load<VEC>(kp + t * p.k_ts + (4 * l + 4 * KL * j));
                    nq[i][j].template load<VEC>(qp + t * q_ts + (4 * l + 4 * KL * j));
                }
                nv[i].template load<VEC>(vp + t * p.v_ts + row0);
            }
        };
        const float A = p.A_log ? -expf(p.A_log[h]) : 0.0f;
        const float bias = p.dt_bias ? ld_io(p.dt_bias, h, p.bias_dtype) : 0.0f;
        DeltaGate gates;  // of token 64 m + lane
        auto gate64 = [&](int t0) {
            const int64_t t = BLK == 1 ? 0 : min(t0 + lane, len - 1);
            gates = delta_gate(p, A, bias, ld_io(p.a, b * p.a_bs + t * p.a_ts + h, p.gate_dtype),
                               ld_io(p.b, b * p.b_bs + t * p.b_ts + h, p.gate_dtype));
        };
        load(0);
        gate64(0);

        float S[R][KE];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float t[4];
                cvt_raw4<ST>(w[r][j], t);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    S[r][4 * j + e] = t[e];
            }

        for (int t0 = 0; t0 < len; t0 += BLK) {
            DeltaRun<IO, 4> ck[BLK][N], cq[BLK][N];
            DeltaRun<IO, R> cv[BLK];
#pragma unroll
            for (int i = 0; i < BLK; ++i) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    ck[i][j] = nk[i][j];
                    ck[i][j].arrive();
                    cq[i][j] = nq[i][j];
                    cq[i][j].arrive();
                }
                cv[i] = nv[i];
                cv[i].arrive();
            }
            if (BLK > 1 && t0 + BLK < len)
                load(t0 + BLK);
            if (BLK > 1 && t0 > 0 && t0 % 64 == 0)
                gate64(t0);
#pragma unroll
            for (int i = 0; i < BLK; ++i) {
                const int t = t0 + i;
                if (BLK > 1 && t >= len)
                    break;
                DeltaGate gate = gates;
                if (BLK > 1) {
                    gate.alpha = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(gates.alpha), t & 63));
                    gate.beta = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(gates.beta), t & 63));
                }
                float kc[KE], qc[KE];
                float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
                for (int e = 0; e < KE; ++e) {
                    kc[e] = ck[i][e / 4][e % 4];
                    qc[e] = cq[i][e / 4][e % 4];
                    kk += kc[e] * kc[e];
                    qq += qc[e] * qc[e];
                    kq += kc[e] * qc[e];
                }
                kk = row_group_sum<KL>(kk);
                qq = row_group_sum<KL>(qq);
                kq = row_group_sum<KL>(kq);
                // v_rsq_f32: within an ulp
                const float rk = p.use_l2 ? __builtin_amdgcn_rsqf(kk + kDeltaEps) : 1.0f;
                const float rq = p.use_l2 ? p.scale * __builtin_amdgcn_rsqf(qq + kDeltaEps) : p.scale;
                kq *= rk;  // of the normalised k, q still as it came
                float o[R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float sk = 0.0f, sq = 0.0f;
#pragma unroll
                    for (int e = 0; e < KE; ++e) {
                        sk += S[r][e] * kc[e];
                        sq += S[r][e] * qc[e];
                    }
                    sk = row_group_sum<KL>(sk);
                    sq = row_group_sum<KL>(sq);
                    const float u = gate.beta * (cv[i][r] - gate.alpha * (sk * rk));
                    const float uk = u * rk;
#pragma unroll
                    for (int e = 0; e < KE; ++e)
                        S[r][e] = S[r][e] * gate.alpha + uk * kc[e];
                    o[r] = (gate.alpha * sq + u * kq) * rq;
                }
                if (outs && l == 0)
                    delta_st_run<IO, R, VEC>(op + (int64_t)t * p.out_ts + row0, o);
            }
        }
        if (p.update) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float t[4] = {S[r][4 * j], S[r][4 * j + 1], S[r][4 * j + 2], S[r][4 * j + 3]};
                    delta_st_state(state + s_off + r * D + 4 * KL * j, t);
                }
        }
    }
    if (outs && l == 0) {
        const float zero[R] = {};
        for (int t = len; t < p.seq_len; ++t)
            delta_st_run<IO, R, VEC>(op + (int64_t)t * p.out_ts + row0, zero);
    }
}

template <typename IO, typename ST, int D, int R>
hipError_t launch_delta_rows_r(const DeltaParams &p, hipStream_t stream)
{
    constexpr int G = 64 / DeltaLanes<D>::KL, TILES = D / (G * R);
    const __int128 waves = (__int128)p.batch * p.hv * TILES;
    const __int128 groups = (waves + 3) / 4;
    if (!launchable(groups, 256))
        return hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)groups);
    constexpr int BLK = D > 128 || sizeof(IO) == 4 ? 2 : 4;  // as the registers of two waves a SIMD allow
    const bool vec = delta_rows_aligned(p, 4 * sizeof(IO));
    if (p.seq_len == 1 && vec)
        delta_rows_kernel<IO, ST, D, R, 1, true><<<grid, 256, 0, stream>>>(p);
    else if (vec)
        delta_rows_kernel<IO, ST, D, R, BLK, true><<<grid, 256, 0, stream>>>(p);
    else
        delta_rows_kernel<IO, ST, D, R, BLK, false><<<grid, 256, 0, stream>>>(p);
    return hipGetLastError();
}

template <typename IO, typename ST>
hipError_t launch_delta_rows_d(const DeltaParams &p, hipStream_t stream)
{
    switch (p.d) {
    case 32: return launch_delta_rows_r<IO, ST, 32, 2>(p, stream);
    case 64: return launch_delta_rows_r<IO, ST, 64, 4>(p, stream);
    case 128: return launch_delta_rows_r<IO, ST, 128, 4>(p, stream);
    default: return launch_delta_rows_r<IO, ST, 256, 4>(p, stream);
    }
}

template <typename IO>
hipError_t launch_delta_rows_io(const DeltaParams &p, hipStream_t stream)
{
    switch (p.state_dtype) {
    case kF32: return launch_delta_rows_d<IO, float>(p, stream);
    case kF16: return launch_delta_rows_d<IO, _Float16>(p, stream);
    default: return launch_delta_rows_d<IO, bf16_t>(p, stream);
    }
}

}  // namespace
}  // namespace ssu
