// The gated delta rule token by token: single tokens, windows of drafted
// tokens, short prompts, and what the matrix cores do not take (fp32
// activations, unaligned rows, head_dim 32 and 256).
//
//   S <- alpha S;  u = beta (v - S k);  S <- S + u k^T;  o = scale S q
//
// A value row of S (D keys) is independent of the others given k. KL lanes
// share a row, each with D / KL of its keys in runs of four (run j of lane l:
// keys 4 (l + KL j) .. + 3, so that one load instruction takes whole lines of
// the pool), and hold R rows. Both products of a token are taken with the
// state before it, o = scale (alpha S_old q + u (k . q)): they run side by
// side, and the chain from a token to the next is one product, its sum over KL
// lanes by DPP, and one multiply-add. The norms of q and k and their product
// are sums over the same lanes.
#pragma once

#include "ssu_delta_impl.h"

namespace ssu {
namespace {

// keys per lane KE = D / KL
template <int D>
struct DeltaLanes {
    static constexpr int KL = D >= 128 ? 16 : D / 8;
    static constexpr int KE = D / KL;
};

// KE entries of a row of q or k for lane l of its KL
template <typename IO, int D, bool VEC>
__device__ __forceinline__ void delta_ld_keys(const void *p, int64_t at, int l,
                                              float (&v)[DeltaLanes<D>::KE])
{
    constexpr int KL = DeltaLanes<D>::KL, KE = DeltaLanes<D>::KE;
#pragma unroll
    for (int j = 0; j < KE / 4; ++j) {
        const int64_t i = at + 4 * (l + KL * j);
        float t[4];
        if constexpr (VEC) {
            cvt_raw4<IO>(ld_raw4<IO>(p, i), t);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                t[e] = ld_elem<IO>(p, i + e);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[4 * j + e] = t[e];
    }
}

// One wave: rows [row0, row0 + G R) of value head h of batch entry b.
template <typename IO, typename ST, int D, int R, bool VEC>
__global__ __launch_bounds__(256) void delta_rows_kernel(DeltaParams p)
{
    constexpr int KL = DeltaLanes<D>::KL, KE = DeltaLanes<D>::KE;
    constexpr int G = 64 / KL;                        // rows side by side in a wave
    constexpr int TILES = D > G * R ? D / (G * R) : 1;  // waves a head
    static_assert(D % (G * R) == 0 || G * R > D, "rows of a head");
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t bh = wave / TILES;
    if (bh >= (int64_t)p.batch * p.hv)
        return;
    const int b = (int)(bh / p.hv), h = (int)(bh - (int64_t)b * p.hv);
    const int l = lane & (KL - 1), row0 = (int)(wave - bh * TILES) * G * R + lane / KL;
    const int pool = p.idx ? p.idx[b] : b;
    const int len = pool < 0 ? 0 : (p.ctx ? clamp_len(p.ctx[b], p.seq_len) : p.seq_len);
    const int jq = h / (p.hv / p.hq);

    float S[R][KE];
    ST *state = nullptr;
    if (len > 0) {
        state = static_cast<ST *>(p.state) + pool * p.row_stride + (int64_t)h * D * D;
        typename Raw4<ST>::type w[R][KE / 4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < KE / 4; ++j)
                w[r][j] = __builtin_nontemporal_load(reinterpret_cast<const typename Raw4<ST>::type *>(
                    state + (row0 + r * G) * D + 4 * (l + KL * j)));
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < KE / 4; ++j) {
                float t[4];
                cvt_raw4<ST>(w[r][j], t);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    S[r][4 * j + e] = t[e];
            }
    }
    const float A = p.A_log && len > 0 ? -expf(p.A_log[h]) : 0.0f;
    const float bias = p.dt_bias && len > 0 ? ld_io(p.dt_bias, h, p.bias_dtype) : 0.0f;
    const int64_t qb = b * p.q_bs + jq * D, kb = b * p.k_bs + jq * D;
    const int64_t vb = b * p.v_bs + h * D, ob = b * p.out_bs + h * D;

    float q[KE] = {}, k[KE] = {}, v[R] = {}, ga = 0.0f, gb = 0.0f;
    auto load = [&](int t) {
        delta_ld_keys<IO, D, VEC>(p.k, kb + t * p.k_ts, l, k);
        if (p.out)
            delta_ld_keys<IO, D, VEC>(p.q, qb + t * p.q_ts, l, q);
#pragma unroll
        for (int r = 0; r < R; ++r)
            v[r] = ld_elem<IO>(p.v, vb + t * p.v_ts + row0 + r * G);
        ga = ld_io(p.a, b * p.a_bs + t * p.a_ts + h, p.gate_dtype);
        gb = ld_io(p.b, b * p.b_bs + t * p.b_ts + h, p.gate_dtype);
    };
    if (len > 0)
        load(0);
    for (int t = 0; t < len; ++t) {
        float qc[KE], kc[KE], vc[R];
#pragma unroll
        for (int e = 0; e < KE; ++e)
            qc[e] = q[e], kc[e] = k[e];
#pragma unroll
        for (int r = 0; r < R; ++r)
            vc[r] = v[r];
        const DeltaGate gate = delta_gate(p, A, bias, ga, gb);
        if (t + 1 < len)
            load(t + 1);
        float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
        for (int e = 0; e < KE; ++e) {
            kk += kc[e] * kc[e];
            qq += qc[e] * qc[e];
            kq += kc[e] * qc[e];
        }
        kk = row_group_sum<KL>(kk);
        qq = row_group_sum<KL>(qq);
        kq = row_group_sum<KL>(kq);
        const float rk = p.use_l2 ? 1.0f / sqrtf(kk + kDeltaEps) : 1.0f;
        const float rq = p.use_l2 ? p.scale / sqrtf(qq + kDeltaEps) : p.scale;
        kq *= rk;  // of the normalised k, q still as it came
        float o = 0.0f;
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
            const float u = gate.beta * (vc[r] - gate.alpha * (sk * rk));
            const float uk = u * rk;
#pragma unroll
            for (int e = 0; e < KE; ++e)
                S[r][e] = S[r][e] * gate.alpha + uk * kc[e];
            const float y = (gate.alpha * sq + u * kq) * rq;
            o = l == r ? y : o;
        }
        if (p.out && l < R)
            st_elem<IO>(p.out, ob + t * p.out_ts + row0 + l * G, o);
    }
    if (p.update && len > 0) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < KE / 4; ++j) {
                const float t[4] = {S[r][4 * j], S[r][4 * j + 1], S[r][4 * j + 2], S[r][4 * j + 3]};
                delta_st_state(state + (row0 + r * G) * D + 4 * (l + KL * j), t);
            }
    }
    if (p.out && l < R)
        for (int t = len; t < p.seq_len; ++t)
            st_elem<IO>(p.out, ob + t * p.out_ts + row0 + l * G, 0.0f);
}

template <typename IO, typename ST, int D, int R>
hipError_t launch_delta_rows_r(const DeltaParams &p, hipStream_t stream)
{
    constexpr int G = 64 / DeltaLanes<D>::KL;
    constexpr int TILES = D > G * R ? D / (G * R) : 1;
    const __int128 waves = (__int128)p.batch * p.hv * TILES;
    const __int128 groups = (waves + 3) / 4;
    if (!launchable(groups, 256))
        return hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)groups);
    if (delta_rows_aligned(p, 4 * sizeof(IO)))
        delta_rows_kernel<IO, ST, D, R, true><<<grid, 256, 0, stream>>>(p);
    else
        delta_rows_kernel<IO, ST, D, R, false><<<grid, 256, 0, stream>>>(p);
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
