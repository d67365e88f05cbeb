// The gated delta rule in chunks of 64 tokens on the matrix cores, for bf16 and
// fp16 activations.
//
// From the state S0 in front of a chunk, with gamma(t, s) the product of the
// decays of tokens s + 1 .. t of the chunk and gamma_t = gamma(t, -1):
//   X_t = beta_t (v_t - gamma_t S0 k_t)
//   U_t = X_t - sum_{s<t} L_ts U_s,       L_ts = beta_t gamma(t, s) (k_t . k_s)
//   o_t = gamma_t S0 q_t + sum_{s<=t} P_ts U_s,  P_ts = gamma(t, s) (q_t . k_s)
//   S   = gamma_C S0 + sum_s gamma(C, s) U_s k_s^T
// Two launches. `prep`, every chunk for itself: L and P in 16 x 16 tiles, and
// the inverses of the diagonal tiles (I + L_ii)^-1 by forward substitution in
// fp32. `sweep`, chunk after chunk: a wave owns 16 value columns of the state and
// needs nothing of the others, so there is no exchange between waves; U comes
// tile after tile (U_i = (I + L_ii)^-1 (X_i - sum_{j<i} L_ij U_j)).
//
// Precision: v_mfma_f32_16x16x32_f16 throughout, fp32 sums. k and q, scaled by a power of
// two to a length in [1, 2), are fp16 exactly but for what lies 2^-25 below
// that length. L, P, the inverses, X, U and the state are pairs of fp16, hi +
// lo, 22 bits: their products keep fp32's accuracy to two bits, the state itself stays
// in fp32 registers. For X, U and the state every value column has a power of
// two of its own, from z = max |v| + 12 max |S| of the column (|S k| <= 12 max |S| at
// 128 keys; 8.5 at 64): z in (2^5, 2^8]. With beta |k|^2 <= 1 a token only shrinks what is
// there and adds its v, so |U| <= 65 z < 2^15; up to 2.1 it grows by 1.1 at most, 64 of
// them by 2^9, and z stays in (2, 2^4]. What is cut off is 2^-25 of these units, 2^-30 of z.
// That is too much where strong decays leave nothing of a state, or of a v, that set the
// scale: with gamma_C < 2^-8 and a v of 16 tokens 2^-8 below z the chunk is not taken.
// A chunk with other values (without the norm; growing decays; a NaN or an infinity)
// is marked by prep, or seen by the wave, and runs token by token in the same
// registers, so that nothing reaches a token before it.
//
// Decays: sums of logarithms only ever add (from a token to its tile's ends, and
// whole tiles between), never subtract, so a log decay of -inf or a far one costs its
// neighbours nothing.
//
// Layouts (lane = 16 g + c): an accumulator tile has column c, rows 4 g + r; an operand
// has row or column c and eight contraction slots of lane group g. The order
// of a contraction's slots is free if both operands have the same, so an
// accumulator serves as an operand as it is: slots 4 g + r of one tile, then of the next (32
// deep), or hi, then lo of one tile (16 deep: [A_hi | A_lo] with [B_hi | B_hi]
// and [B_lo | 0], both products in two instructions). S^T [key][value] is such an
// accumulator: it never leaves registers. K is kept with its keys in that
// order, in two planes of 8 bytes a lane, which both a row read (two planes) and
// a transposed read (ds_read_b64_tr_b16, one plane) take without bank conflicts.
#pragma once

#include "ssu_delta_impl.h"

namespace ssu {
namespace {

constexpr int kDcC = 64;          // tokens of a chunk
constexpr int kDcTile = 1024;     // bytes of an inverse as [hi | lo], or of a plane (hi or lo) of two tiles
// Block of a value head and chunk: 4 inverses, 4 pairs of tiles of L (the second of rows
// 1 and 3's last is zero), scalars, 6 pairs of P (what lies above the diagonal is zero)
constexpr int kDcL = 4 * kDcTile, kDcScalars = 12 * kDcTile, kDcP = 14 * kDcTile;
constexpr int kDcHead = kDeltaHeadBytes;
static_assert(kDcHead == 26 * kDcTile, "tiles of a head");
__device__ __forceinline__ constexpr int dc_l_pair(int i, int p) { return kDcL + (i - 1 + p) * 2 * kDcTile; }
__device__ __forceinline__ constexpr int dc_p_pair(int i, int p)
{
    return kDcP + (i < 2 ? i : 2 * i - 2 + p) * 2 * kDcTile;
}
// Scalars: arrays of 64 floats
enum : int { kScBeta, kScGk, kScWk, kScAlpha, kScKs, kScGo, kScQo, kScMisc };

typedef _Float16 dc_f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 dc_f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 dc_f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 dc_bf16x2 __attribute__((ext_vector_type(2)));
typedef float dc_f32x2 __attribute__((ext_vector_type(2)));
typedef float dc_f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t dc_u16x2 __attribute__((ext_vector_type(2)));
typedef short dc_i16x4 __attribute__((ext_vector_type(4)));

struct DeltaWork {
    unsigned char *kq;     // [batch][chunks][Hq]: K, then Q of 64 tokens
    unsigned char *head;   // [batch][chunks][HV][kDcHead]
    float *carry;          // [batch][HV][D][D] between segments
    int chunk0, chunks;    // the segment
    int first, last;       // of all segments
};

__device__ __forceinline__ dc_f32x4 dc_mfma(const u32x4 &a, const u32x4 &b, const dc_f32x4 &c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(dc_f16x8, a),
                                                  __builtin_bit_cast(dc_f16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ dc_f32x4 dc_mfma16(const u32x2 &a, const u32x2 &b, const dc_f32x4 &c)
{
    return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(dc_f16x4, a),
                                                 __builtin_bit_cast(dc_f16x4, b), c, 0, 0, 0);
}

// Four fp32 values as fp16 pairs: hi (2 words) and what is left (2 words). The factor -1
// comes from a register, so that the difference is one v_fma_mix_f32, which
// takes the fp16 as it is.
__device__ __forceinline__ void dc_split(const dc_f32x4 &f, u32x2 &hi, u32x2 &lo)
{
    float minus;
    asm("v_mov_b32 %0, -1.0" : "=v"(minus));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float a = f[2 * e], b = f[2 * e + 1];
        const dc_f16x2 h = __builtin_convertvector((dc_f32x2){a, b}, dc_f16x2);
        const dc_f16x2 l = __builtin_convertvector(
            (dc_f32x2){fmaf((float)h[0], minus, a), fmaf((float)h[1], minus, b)}, dc_f16x2);
        hi[e] = __builtin_bit_cast(uint32_t, h);
        lo[e] = __builtin_bit_cast(uint32_t, l);
    }
}

// Two values rounded to nearest even in a 16-bit type
template <typename IO>
__device__ __forceinline__ uint32_t dc_pack(float a, float b)
{
    if constexpr (__is_same(IO, _Float16))
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((dc_f32x2){a, b}, dc_f16x2));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((dc_f32x2){a, b}, dc_bf16x2));
}

// Byte offset in a K or Q image of the 8 bytes with keys 16 n + 4 g .. + 3 of token `tok`
template <int D>
__device__ __forceinline__ int dc_at(int tok, int n, int g)
{
    return (((tok >> 4) * (D / 32) + (n >> 1)) * 2 + (n & 1)) * 512 + (g * 16 + (tok & 15)) * 8;
}

// An operand of 32 keys (step ks) of the 16 tokens of tile i, or any two planes
template <int D>
__device__ __forceinline__ u32x4 dc_ld_op(const unsigned char *image, int i, int ks, int lane)
{
    const unsigned char *p = image + (i * (D / 32) + ks) * 1024 + lane * 8;
    const u32x2 a = *reinterpret_cast<const u32x2 *>(p);
    const u32x2 b = *reinterpret_cast<const u32x2 *>(p + 512);
    return u32x4{a[0], a[1], b[0], b[1]};
}

template <int LANE>
__device__ __forceinline__ float dc_bcast16(float v)  // lane LANE of the own row of 16
{
    return dpp_f32<0x150 + LANE>(v);
}

// D[t][.] -= L[t][M] D[M][.] for M = 0 .. 14: row M is final when its turn comes
template <int M>
__device__ __forceinline__ void dc_invert(const float (&L)[16], dc_f32x4 &d)
{
    if constexpr (M < 15) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            d[r] -= L[M] * dc_bcast16<M>(d[r]);
        dc_invert<M + 1>(L, d);
    }
}

// Sums over the four lane groups (lanes c, c + 16, c + 32, c + 48)
__device__ __forceinline__ float dc_sum_groups(float v)
{
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
__device__ __forceinline__ uint32_t dc_max_groups(uint32_t v)
{
    const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max((uint32_t)a[0], (uint32_t)a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return max((uint32_t)b[0], (uint32_t)b[1]);
}

// Gates of one value head and chunk that prep's waves share
struct DcGates {
    float beta[kDcC];   // beta_t k_s(t): of the fp16 keys
    float row[kDcC];    // decay from the tile's start through t
    float tail[kDcC];   // decay behind t to the tile's end, times k_s(t)
    float log[kDcC];
    float total[4];     // logs of a tile
};

template <typename IO, int D>
struct DcPrepLds {
    unsigned char k[kDcC * D * 2], q[kDcC * D * 2];
    float ks[kDcC], qs[kDcC], kk[kDcC];  // length of k as fp16 -> k; of q -> scaled q; |k|^2
    float qq[kDcC];
    DcGates gates[4];
    float diag[4][16 * 20];
};

template <typename IO, int D>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaParams p, DeltaWork w)
{
    constexpr int KS = D / 32;
    __shared__ DcPrepLds<IO, D> lds;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int G = p.hv / p.hq;
    const int chunk = blockIdx.x / p.hq, j = blockIdx.x - chunk * p.hq, b = blockIdx.y;
    const int pool = p.idx ? p.idx[b] : b;
    const int len = pool < 0 ? 0 : (p.ctx ? clamp_len(p.ctx[b], p.seq_len) : p.seq_len);
    const int t0 = (w.chunk0 + chunk) * kDcC;
    const int n = min(len - t0, kDcC);
    if (n <= 0) {
        if (p.out) {
            const int to = min(p.seq_len - t0, kDcC), words = G * D / 4;
            uint16_t *o = static_cast<uint16_t *>(p.out) + b * p.out_bs + (int64_t)j * G * D;
            for (int i = threadIdx.x; i < to * words; i += 256) {
                const int t = i / words;
                *reinterpret_cast<u32x2 *>(o + (t0 + t) * p.out_ts + 4 * (i - t * words)) = u32x2{0, 0};
            }
        }
        return;
    }

    // k and q of tile `wave`: lengths, fp16
    {
        const int tok = 16 * wave + c;
        const bool in = tok < n;
        const uint16_t *kp = static_cast<const uint16_t *>(p.k) + b * p.k_bs + (t0 + tok) * p.k_ts + j * D + 8 * g;
        const uint16_t *qp = static_cast<const uint16_t *>(p.q) + b * p.q_bs + (t0 + tok) * p.q_ts + j * D + 8 * g;
        u32x4 raw[2][KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            raw[0][ks] = raw[1][ks] = u32x4{0, 0, 0, 0};
            if (in) {
                raw[0][ks] = *reinterpret_cast<const u32x4 *>(kp + 32 * ks);
                if (p.out)
                    raw[1][ks] = *reinterpret_cast<const u32x4 *>(qp + 32 * ks);
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float v[KS][8], sum = 0.0f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[ks][e] = cvt_raw1<IO>(e % 2 ? raw[s][ks][e / 2] >> 16 : raw[s][ks][e / 2] & 0xffffu);
                    sum += v[ks][e] * v[ks][e];
                }
            sum = dc_sum_groups(sum);
            const bool fine = sum > 0.0f && sum < __builtin_inff();
            const int ex = fine ? min(max(1 - __builtin_amdgcn_frexp_expf(sqrtf(sum)), -126), 126) : 0;
            const float up = __builtin_amdgcn_ldexpf(1.0f, ex), down = __builtin_amdgcn_ldexpf(1.0f, -ex);
            unsigned char *image = s ? lds.q : lds.k;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    h[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(
                        (dc_f32x2){v[ks][2 * e] * up, v[ks][2 * e + 1] * up}, dc_f16x2));
                // keys 32 ks + 8 g ..: pieces 2 g and 2 g + 1 of the eight pieces of a step
                *reinterpret_cast<u32x2 *>(image + dc_at<D>(tok, 2 * ks + (g >> 1), 2 * (g & 1))) = u32x2{h[0], h[1]};
                *reinterpret_cast<u32x2 *>(image + dc_at<D>(tok, 2 * ks + (g >> 1), 2 * (g & 1) + 1)) = u32x2{h[2], h[3]};
            }
            const float r = p.use_l2 ? 1.0f / sqrtf(sum + kDeltaEps) : 1.0f;
            if (g == 0) {
                if (s == 0) {
                    lds.ks[tok] = r * down;
                    lds.kk[tok] = sum * r * r;  // NaN or inf where k's is
                } else {
                    lds.qs[tok] = r * down * p.scale;
                    lds.qq[tok] = sum;
                }
            }
        }
    }
    __syncthreads();
    const int64_t at = (int64_t)b * w.chunks + chunk;
    {
        unsigned char *to = w.kq + (at * p.hq + j) * (4 * kDcC * D);
#pragma unroll
        for (int i = 0; i < kDcC * D * 2 / 4096; ++i) {
            const int o = (i * 256 + threadIdx.x) * 16;
            *reinterpret_cast<u32x4 *>(to + o) = *reinterpret_cast<const u32x4 *>(lds.k + o);
            if (p.out)
                *reinterpret_cast<u32x4 *>(to + 2 * kDcC * D + o) = *reinterpret_cast<const u32x4 *>(lds.q + o);
        }
    }

    // K_s . K_t of row tile `wave`, K_s . Q_t of row tile 3 - wave (five tiles a wave): column
    // t of the tile, rows s
    const int ip = 3 - wave;
    dc_f32x4 kk[4], qk[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        kk[t] = qk[t] = dc_f32x4{0, 0, 0, 0};
        if (t <= wave)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                kk[t] = dc_mfma(dc_ld_op<D>(lds.k, t, ks, lane), dc_ld_op<D>(lds.k, wave, ks, lane), kk[t]);
        if (p.out && t <= ip)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                qk[t] = dc_mfma(dc_ld_op<D>(lds.k, t, ks, lane), dc_ld_op<D>(lds.q, ip, ks, lane), qk[t]);
    }

    for (int h0 = 0; h0 < G; h0 += 4) {
        if (h0 + wave < G) {  // gates of four heads at once, lane = token
            const int h = j * G + h0 + wave;
            const bool in = lane < n;
            float lg = 0.0f, beta = 0.0f;
            if (in) {
                const float A = p.A_log ? -expf(p.A_log[h]) : 0.0f;
                const float bias = p.dt_bias ? ld_io(p.dt_bias, h, p.bias_dtype) : 0.0f;
                const int64_t t = t0 + lane;
                lg = delta_log_decay(p, A, bias, ld_io(p.a, b * p.a_bs + t * p.a_ts + h, p.gate_dtype));
                beta = delta_beta(p, ld_io(p.b, b * p.b_bs + t * p.b_ts + h, p.gate_dtype));
            }
            const float ks = lds.ks[lane], qs = lds.qs[lane], kk2 = lds.kk[lane];
            const bool bad = in && !(lg <= 0.0f && kk2 <= 1.07f && fabsf(beta) * kk2 <= 2.1f &&
                                     (!p.out || lds.qq[lane] < __builtin_inff()));
            const bool wide = in && !(beta >= 0.0f && beta <= 1.02f && beta * kk2 <= 1.02f);
            const float kind = __ballot(bad) ? 1.0f : __ballot(wide) ? 2.0f : 0.0f;
            const float row = row_prefix_sum16(lg);
            // behind the token to its tile's end: the suffix sum of the next token
            const float tail = dpp_f32_fill<0x101>(0.0f, row_suffix_sum16(lg));
            float total[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                total[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, row), 16 * i + 15));
            float before = 0.0f, behind = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                before += i < g ? total[i] : 0.0f;
                behind += i > g ? total[i] : 0.0f;
            }
            DcGates &s = lds.gates[wave];
            s.beta[lane] = beta * ks;
            s.row[lane] = expf(row);
            s.tail[lane] = expf(tail) * ks;
            s.log[lane] = lg;
            if (lane < 4)
                s.total[lane] = lane == 0 ? total[0] : lane == 1 ? total[1] : lane == 2 ? total[2] : total[3];
            float *sc = reinterpret_cast<float *>(w.head + (at * p.hv + h) * kDcHead + kDcScalars);
            const float gamma = expf(before + row);
            sc[kScBeta * 64 + lane] = beta;
            sc[kScGk * 64 + lane] = gamma * ks;
            sc[kScWk * 64 + lane] = expf(behind + tail) * ks;
            sc[kScAlpha * 64 + lane] = expf(lg);
            sc[kScKs * 64 + lane] = ks;
            sc[kScGo * 64 + lane] = gamma * qs;
            sc[kScQo * 64 + lane] = qs;
            const float all = expf((total[0] + total[1]) + (total[2] + total[3]));
            sc[kScMisc * 64 + lane] = lane == 0 ? all : lane == 1 ? kind : 0.0f;
        }
        __syncthreads();
        for (int hh = 0; hh < 4 && h0 + hh < G; ++hh) {
            const DcGates &s = lds.gates[hh];
            unsigned char *to = w.head + (at * p.hv + j * G + h0 + hh) * kDcHead;
            // both kinds of tiles: L of row tile `wave`, P of row tile ip
#pragma unroll
            for (int kind = 0; kind < 2; ++kind) {
                if (kind == 1 && !p.out)
                    break;
                const int i = kind ? ip : wave;
                const int t = 16 * i + c;
                const float own = kind ? 1.0f : s.beta[t];
                const float front = -own * s.row[t];  // L is stored with its sign in U's recursion
#pragma unroll
                for (int jt = 0; jt < 3; ++jt) {
                    if (jt >= i)
                        break;
                    float mid = 0.0f;
                    for (int m = jt + 1; m < i; ++m)
                        mid += s.total[m];
                    const float f = (kind ? -front : front) * expf(mid);
                    const dc_f32x4 tail = *reinterpret_cast<const dc_f32x4 *>(&s.tail[16 * jt + 4 * g]);
                    dc_f32x4 v;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        v[r] = f * ((kind ? qk[jt][r] : kk[jt][r]) * tail[r]);
                    u32x2 hi, lo;
                    dc_split(v, hi, lo);
                    unsigned char *at8 = to + (kind ? dc_p_pair(i, jt >> 1) : dc_l_pair(i, jt >> 1)) + lane * 16 + 8 * (jt & 1);
                    *reinterpret_cast<u32x2 *>(at8) = hi;
                    *reinterpret_cast<u32x2 *>(at8 + kDcTile) = lo;
                }
                // diagonal tile: decays behind s through t by adding from t downwards
                float sum = 0.0f;
                dc_f32x4 dl = {0, 0, 0, 0};
                for (int m = 15; m >= 1; --m) {
                    sum += m <= c ? s.log[16 * i + m] : 0.0f;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        dl[r] = 4 * g + r == m - 1 ? sum : dl[r];
                }
                dc_f32x4 v;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int ss = 4 * g + r;
                    float x = kind ? qk[3][r] : kk[3][r];
#pragma unroll
                    for (int q = 0; q < 3; ++q)
                        x = i == q ? (kind ? qk[q][r] : kk[q][r]) : x;
                    const float d = expf(dl[r]) * lds.ks[16 * i + ss] * own * x;
                    v[r] = ss < c || (kind && ss == c) ? d : 0.0f;
                }
                if (kind == 0) {
                    float *tile = lds.diag[wave];
                    __builtin_amdgcn_wave_barrier();
                    *reinterpret_cast<dc_f32x4 *>(tile + c * 20 + 4 * g) = v;
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                    float L[16];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const dc_f32x4 x = *reinterpret_cast<const dc_f32x4 *>(tile + c * 20 + 4 * q);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            L[4 * q + r] = x[r];
                    }
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        v[r] = 4 * g + r == c ? 1.0f : 0.0f;
                    dc_invert<0>(L, v);
                }
                u32x2 hi, lo;
                dc_split(v, hi, lo);
                if (kind == 0) {
                    *reinterpret_cast<u32x4 *>(to + i * kDcTile + lane * 16) = u32x4{hi[0], hi[1], lo[0], lo[1]};
                    if (i & 1) {  // the second tile of this row's last pair
                        unsigned char *at8 = to + dc_l_pair(i, i >> 1) + lane * 16 + 8;
                        *reinterpret_cast<u32x2 *>(at8) = *reinterpret_cast<u32x2 *>(at8 + kDcTile) = u32x2{0, 0};
                    }
                } else {
                    unsigned char *at8 = to + dc_p_pair(i, i >> 1) + lane * 16 + 8 * (i & 1);
                    *reinterpret_cast<u32x2 *>(at8) = hi;
                    *reinterpret_cast<u32x2 *>(at8 + kDcTile) = lo;
                    if (!(i & 1))
                        *reinterpret_cast<u32x2 *>(at8 + 8) = *reinterpret_cast<u32x2 *>(at8 + kDcTile + 8) = u32x2{0, 0};
                }
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------

typedef __attribute__((address_space(3))) dc_i16x4 *dc_lds_v4;

// 16 bytes a lane from global memory to LDS: `to` is the wave's, lane i's land at to + 16 i.
// In assembly, as with the builtin the compiler waits for these loads in front of the
// next LDS read of any address; they are waited for once a chunk, by hand. No register
// receives anything. The addresses of lanes are read at issue.
__device__ __forceinline__ void dc_to_lds(const unsigned char *from, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(to), "v"(from)
                 : "memory", "m0");
}

// K^T operand: rows keys 16 n + c, contraction the tokens 16 i + 4 g + r of tiles i = 2 s, 2 s + 1
template <int D>
__device__ __forceinline__ u32x4 dc_ld_kt(unsigned char *image, int n, int s, int lane)
{
    const int g = lane >> 4, x = lane & 15;
    unsigned char *p = image + dc_at<D>(32 * s + 4 * g + (x >> 2), n, x & 3);
    const dc_i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((dc_lds_v4)p);
    const dc_i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((dc_lds_v4)(p + (D / 32) * 1024));
    const u32x2 a2 = __builtin_bit_cast(u32x2, a), b2 = __builtin_bit_cast(u32x2, b);
    return u32x4{a2[0], a2[1], b2[0], b2[1]};
}

// Values of token rows in LDS: four tokens 4 g + r of tile i, column c of the wave's (as bits)
template <int PITCH>
__device__ __forceinline__ u32x2 dc_ld_v(unsigned char *rows, int i, int lane)
{
    const int g = lane >> 4, x = lane & 15;
    unsigned char *p = rows + (16 * i + 4 * g + (x >> 2)) * PITCH + (x & 3) * 8;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((dc_lds_v4)p));
}

// The largest magnitude of tile maxima m (bits of 16-bit values, two tiles a word) over
// the four lane groups
__device__ __forceinline__ uint32_t dc_max2_groups(uint32_t m)
{
    auto larger = [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(dc_u16x2, a),
                                                                      __builtin_bit_cast(dc_u16x2, b)));
    };
    const auto a = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    m = larger(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    return larger(b[0], b[1]);
}

// One wave: value columns [16 NV (..)] of value head h, batch entry b.
template <typename IO, int D, int NV, int W, bool OUT>
__global__ __launch_bounds__(64 * W, W / 4) void delta_sweep_kernel(DeltaParams p, DeltaWork w, int swizzle)
{
    constexpr int KS = D / 32, KT = D / 16, C = kDcC;
    constexpr int TILES = D / (16 * W * NV);           // workgroups a head
    constexpr int KQ = 4 * C * D, VP = 32 * W * NV;    // bytes of K and Q, of a token's values
    constexpr int BUF = KQ + kDcHead + C * VP;         // of a chunk in LDS
    static_assert(TILES * 16 * W * NV == D, "value columns of a head");
    __shared__ __attribute__((aligned(16))) unsigned char lds[2 * BUF];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    // workgroups are dealt out over eight XCDs: those of one q head go to the same one
    const uint32_t id = swizzle ? (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3) : blockIdx.x;
    const int64_t bh = id / TILES;
    const int b = (int)(bh / p.hv), h = (int)(bh - (int64_t)b * p.hv);
    const int wg_v0 = (int)(id - bh * TILES) * (16 * W * NV), v0 = wg_v0 + wave * 16 * NV;
    const int j = h / (p.hv / p.hq);
    const int pool = p.idx ? p.idx[b] : b;
    const int len = pool < 0 ? 0 : (p.ctx ? clamp_len(p.ctx[b], p.seq_len) : p.seq_len);
    const int mine = min(len - w.chunk0 * C, w.chunks * C);  // tokens of the segment
    if (len <= 0 || (mine <= 0 && !(w.last && p.update && !w.first)))
        return;
    const int chunks = mine > 0 ? (mine + C - 1) / C : 0;

    // What prep left of a chunk, and its values, go to LDS past the registers, 1 KiB an
    // instruction, while the chunk before it is worked on
    const unsigned char *kq = w.kq + ((int64_t)b * w.chunks * p.hq + j) * KQ + lane * 16;
    const unsigned char *hd = w.head + ((int64_t)b * w.chunks * p.hv + h) * kDcHead + lane * 16;
    const int64_t kq_step = (int64_t)p.hq * KQ, hd_step = (int64_t)p.hv * kDcHead;
    constexpr int VL = VP / 16, VR = 64 / VL;  // lanes a token's values, tokens an instruction
    const uint16_t *vp = static_cast<const uint16_t *>(p.v) + b * p.v_bs + (int64_t)w.chunk0 * C * p.v_ts +
                         (int64_t)h * D + wg_v0 + 8 * (lane % VL);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char *)lds;
    // part 0 .. 3 of four (the CU takes 64 bytes a cycle: issued at once, they would stall the wave)
    auto fetch = [&](int ch, int part) {
        uint32_t to = lds0 + (ch & 1) * BUF;
        const unsigned char *from = kq + ch * kq_step;
        constexpr int QK = OUT ? KQ : KQ / 2;
#pragma unroll
        for (int o = 0; o < QK; o += W * 1024)
            if (o / (W * 1024) % 4 == part)
                dc_to_lds(from + o + wave * 1024, to + o + wave * 1024);
        to += KQ;
        from = hd + ch * hd_step;
        constexpr int HD = OUT ? kDcHead : kDcP;
#pragma unroll
        for (int o = 0; o < HD; o += W * 1024)
            if (o / (W * 1024) % 4 == part && (o + W * 1024 <= HD || o + wave * 1024 < HD))
                dc_to_lds(from + o + wave * 1024, to + o + wave * 1024);
        to += kDcHead;
#pragma unroll
        for (int q = 0; q < C / VR; q += W)
            if (q / W % 4 == part) {
                const int t = ch * C + (q + wave) * VR + lane / VL;  // rows behind the end repeat the last
                dc_to_lds(reinterpret_cast<const unsigned char *>(vp + (int64_t)min(t, mine - 1) * p.v_ts),
                          to + (q + wave) * 1024);
            }
    };
    if (chunks > 0)
#pragma unroll
        for (int part = 0; part < 4; ++part)
            fetch(0, part);

    // The state: S^T, tile n of keys; rows (keys) 4 g + r, column (value) c
    dc_f32x4 S[NV][KT];
    const int64_t head_at = pool * p.row_stride + (int64_t)h * D * D;
    float *carry = w.carry + ((int64_t)b * p.hv + h) * D * D;
    if (!w.first || p.state_dtype == kF32) {
        const float *s = (w.first ? static_cast<const float *>(p.state) + head_at : carry) + (v0 + c) * D + 4 * g;
#pragma unroll
        for (int x = 0; x < NV; ++x)
#pragma unroll
            for (int n = 0; n < KT; ++n)
                S[x][n] = *reinterpret_cast<const dc_f32x4 *>(s + 16 * x * D + 16 * n);
    } else {
        const uint16_t *s = static_cast<const uint16_t *>(p.state) + head_at + (v0 + c) * D + 4 * g;
        u32x2 raw[NV][KT];
#pragma unroll
        for (int x = 0; x < NV; ++x)
#pragma unroll
            for (int n = 0; n < KT; ++n)
                raw[x][n] = *reinterpret_cast<const u32x2 *>(s + 16 * x * D + 16 * n);
        auto widen = [&](auto tag) {
#pragma unroll
            for (int x = 0; x < NV; ++x)
#pragma unroll
                for (int n = 0; n < KT; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        S[x][n][r] = cvt_raw1<decltype(tag)>(r % 2 ? raw[x][n][r / 2] >> 16 : raw[x][n][r / 2] & 0xffffu);
        };
        if (p.state_dtype == kF16)
            widen(_Float16{});
        else
            widen(bf16_t{});
    }
    uint16_t *op = static_cast<uint16_t *>(p.out) + b * p.out_bs + (int64_t)h * D + v0;
    const int o_off = c * (int)p.out_ts + 4 * g;
    float sc[NV];        // scale of the value column of this lane
    float isc[NV][4];    // 1 / scale of value columns 4 g + r
#pragma unroll
    for (int x = 0; x < NV; ++x) {
        sc[x] = 1.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            isc[x][r] = 1.0f;
    }

    for (int ch = 0; ch < chunks; ++ch) {
        // this chunk's LDS is filled (by every wave: behind the barrier), the other one read
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        unsigned char *image = lds + (ch & 1) * BUF;
        const unsigned char *blk = image + KQ;
        const float *scal = reinterpret_cast<const float *>(blk + kDcScalars);
        const int t0 = ch * C, n_tok = min(mine - t0, C);
        const int64_t tok0 = (int64_t)w.chunk0 * C + t0;
        const bool more = ch + 1 < chunks;
        if (more)
            fetch(ch + 1, 0);
        u32x2 raw[NV][4];
#pragma unroll
        for (int x = 0; x < NV; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                raw[x][i] = dc_ld_v<VP>(image + KQ + kDcHead + (wave * NV + x) * 32, i, lane);
        if (n_tok < C) {  // what was read in the place of tokens behind the end
#pragma unroll
            for (int x = 0; x < NV; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = 16 * i + 4 * g + 2 * e;
                        raw[x][i][e] &= (t < n_tok ? 0xffffu : 0u) | (t + 1 < n_tok ? 0xffff0000u : 0u);
                    }
        }

        u32x4 kf[4];  // in flight over the scales
#pragma unroll
        for (int i = 0; i < 4; ++i)
            kf[i] = dc_ld_op<D>(image, i, 0, lane);

        // scales, and whether the chunk may run on the matrix cores
        const float all = scal[kScMisc * 64], kind = scal[kScMisc * 64 + 1];
        const float top = kind == 2.0f ? 0x1p4f : 0x1p8f;
        const bool fades = all < 0x1p-8f;
        bool slow = kind == 1.0f;
        bool move = false;
        float z[NV];
#pragma unroll
        for (int x = 0; x < NV; ++x) {
            float ms[2] = {0.0f, 0.0f};  // a NaN of the state reaches every token of the chunk anyway
#pragma unroll
            for (int n = 0; n < KT; ++n)
                ms[n & 1] = fmaxf(fmaxf(fmaxf(ms[n & 1], fabsf(S[x][n][0])), fabsf(S[x][n][1])),
                                  fmaxf(fabsf(S[x][n][2]), fabsf(S[x][n][3])));
            uint32_t tile[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(
                    __builtin_bit_cast(dc_u16x2, raw[x][i][0] & 0x7fff7fffu),
                    __builtin_bit_cast(dc_u16x2, raw[x][i][1] & 0x7fff7fffu)));
                tile[i] = max(m & 0xffffu, m >> 16);
            }
            constexpr uint32_t kInf = __is_same(IO, _Float16) ? 0x7c00u : 0x7f80u;
            const uint32_t mv = max(max(tile[0], tile[1]), max(tile[2], tile[3]));
            slow |= mv >= kInf;
            // z from one exchange: twice the larger of its two parts
            const float part = fmaxf(cvt_raw1<IO>(mv) * sc[x], (D > 64 ? 12.0f : 8.5f) * fmaxf(ms[0], ms[1]));
            z[x] = 2.0f * __uint_as_float(dc_max_groups(__float_as_uint(part)));
            slow |= !(z[x] < __builtin_inff());
            if (fades) {
                const uint32_t m01 = dc_max2_groups(tile[0] | tile[1] << 16);
                const uint32_t m23 = dc_max2_groups(tile[2] | tile[3] << 16);
                uint32_t least = n_tok >= 16 ? m01 & 0xffffu : kInf;  // of whole tiles
                least = n_tok >= 32 ? min(least, m01 >> 16) : least;
                least = n_tok >= 48 ? min(least, m23 & 0xffffu) : least;
                least = n_tok >= 64 ? min(least, m23 >> 16) : least;
                slow |= cvt_raw1<IO>(least) * sc[x] < z[x] * 0x1p-8f;
            }
            move |= z[x] > top || (z[x] <= top * 0x1p-3f && z[x] > 0.0f);
        }
        slow = __ballot(slow) != 0;
        if (!slow && __ballot(move)) {
#pragma unroll
            for (int x = 0; x < NV; ++x) {
                const bool m = z[x] > top || (z[x] <= top * 0x1p-3f && z[x] > 0.0f);
                int k = m ? __builtin_amdgcn_frexp_expf(top) - 1 - __builtin_amdgcn_frexp_expf(z[x]) : 0;
                // the scale itself stays within 2^-124 .. 2^124, which every finite z reaches
                const int e = __builtin_amdgcn_frexp_expf(sc[x]) - 1;
                k = min(max(k, -124 - e), 124 - e);
                const float f = __builtin_amdgcn_ldexpf(1.0f, k);
                sc[x] *= f;
#pragma unroll
                for (int n = 0; n < KT; ++n)
                    S[x][n] *= f;
                const float inv = __builtin_amdgcn_ldexpf(1.0f, -(e + k));
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    isc[x][r] = __shfl(inv, 4 * g + r, 64);
            }
        }

        if (!slow) {
            dc_f32x4 X[NV][4], O[NV][4];
#pragma unroll
            for (int x = 0; x < NV; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    X[x][i] = O[x][i] = dc_f32x4{0, 0, 0, 0};
            // S0 k and S0 q
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                u32x4 sh[NV], sl[NV];
#pragma unroll
                for (int x = 0; x < NV; ++x) {
                    u32x2 h0, l0, h1, l1;
                    dc_split(S[x][2 * ks], h0, l0);
                    dc_split(S[x][2 * ks + 1], h1, l1);
                    sh[x] = u32x4{h0[0], h0[1], h1[0], h1[1]};
                    sl[x] = u32x4{l0[0], l0[1], l1[0], l1[1]};
                }
                u32x4 qf[4], kn[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (OUT)
                        qf[i] = dc_ld_op<D>(image + KQ / 2, i, ks, lane);
                    if (ks + 1 < KS)
                        kn[i] = dc_ld_op<D>(image, i, ks + 1, lane);
                }
#pragma unroll
                for (int x = 0; x < NV; ++x) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        X[x][i] = dc_mfma(kf[i], sh[x], X[x][i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        X[x][i] = dc_mfma(kf[i], sl[x], X[x][i]);
                }
                if (OUT)
#pragma unroll
                    for (int x = 0; x < NV; ++x) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            O[x][i] = dc_mfma(sh[x], qf[i], O[x][i]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            O[x][i] = dc_mfma(sl[x], qf[i], O[x][i]);
                    }
                if (ks + 1 < KS)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        kf[i] = kn[i];
            }
            if (more)
                fetch(ch + 1, 1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const dc_f32x4 beta = *reinterpret_cast<const dc_f32x4 *>(scal + kScBeta * 64 + 16 * i + 4 * g);
                const dc_f32x4 gk = *reinterpret_cast<const dc_f32x4 *>(scal + kScGk * 64 + 16 * i + 4 * g);
#pragma unroll
                for (int x = 0; x < NV; ++x)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                    {
                        const float vt = cvt_raw1<IO>(r % 2 ? raw[x][i][r / 2] >> 16 : raw[x][i][r / 2] & 0xffffu);
                        X[x][i][r] = beta[r] * (vt * sc[x] - gk[r] * X[x][i][r]);
                    }
            }
            if (more)
                fetch(ch + 1, 2);
            // U, tile after tile: 32-deep operands are pairs of tiles
            u32x4 uh[NV][2], ul[NV][2];
#pragma unroll
            for (int x = 0; x < NV; ++x)
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    uh[x][q] = ul[x][q] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int q = 0; 2 * q < i; ++q) {
                    const u32x4 lh = *reinterpret_cast<const u32x4 *>(blk + dc_l_pair(i, q) + lane * 16);
                    const u32x4 ll = *reinterpret_cast<const u32x4 *>(blk + dc_l_pair(i, q) + kDcTile + lane * 16);
#pragma unroll
                    for (int x = 0; x < NV; ++x) {
                        X[x][i] = dc_mfma(ll, uh[x][q], X[x][i]);
                        X[x][i] = dc_mfma(lh, ul[x][q], X[x][i]);
                        X[x][i] = dc_mfma(lh, uh[x][q], X[x][i]);
                    }
                }
                const u32x4 df = *reinterpret_cast<const u32x4 *>(blk + i * kDcTile + lane * 16);
                const u32x2 dh = {df[0], df[1]}, dl = {df[2], df[3]};
#pragma unroll
                for (int x = 0; x < NV; ++x) {
                    u32x2 hi, lo;
                    dc_split(X[x][i], hi, lo);
                    dc_f32x4 u = {0, 0, 0, 0};
                    u = dc_mfma16(dl, hi, u);
                    u = dc_mfma16(dh, lo, u);
                    u = dc_mfma16(dh, hi, u);
                    X[x][i] = u;
                    dc_split(u, hi, lo);
                    uh[x][i >> 1][2 * (i & 1)] = hi[0];
                    uh[x][i >> 1][2 * (i & 1) + 1] = hi[1];
                    ul[x][i >> 1][2 * (i & 1)] = lo[0];
                    ul[x][i >> 1][2 * (i & 1) + 1] = lo[1];
                }
            }
            if (more)
                fetch(ch + 1, 3);
            if (OUT) {
                dc_f32x4 Q[NV][4];
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 2 * r; i < 4; ++i) {
                        const u32x4 ph = *reinterpret_cast<const u32x4 *>(blk + dc_p_pair(i, r) + lane * 16);
                        const u32x4 pl = *reinterpret_cast<const u32x4 *>(blk + dc_p_pair(i, r) + kDcTile + lane * 16);
#pragma unroll
                        for (int x = 0; x < NV; ++x) {
                            if (r == 0)
                                Q[x][i] = dc_f32x4{0, 0, 0, 0};
                            Q[x][i] = dc_mfma(uh[x][r], pl, Q[x][i]);
                            Q[x][i] = dc_mfma(ul[x][r], ph, Q[x][i]);
                            Q[x][i] = dc_mfma(uh[x][r], ph, Q[x][i]);
                        }
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float go = scal[kScGo * 64 + 16 * i + c], qo = scal[kScQo * 64 + 16 * i + c];
#pragma unroll
                    for (int x = 0; x < NV; ++x) {
                        float o[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            o[r] = isc[x][r] * (go * O[x][i][r] + qo * Q[x][i][r]);
                        const u32x2 bits = {dc_pack<IO>(o[0], o[1]), dc_pack<IO>(o[2], o[3])};
                        u32x2 *to = reinterpret_cast<u32x2 *>(op + (tok0 + 16 * i) * p.out_ts + (o_off + 16 * x));
                        if (n_tok == C) {
                            *to = bits;
                        } else if (tok0 + 16 * i + c < p.seq_len) {
                            *to = 16 * i + c < n_tok ? bits : u32x2{0, 0};
                        }
                    }
                }
            }
            // the state behind the chunk
#pragma unroll
            for (int x = 0; x < NV; ++x)
#pragma unroll
                for (int n = 0; n < KT; ++n)
                    S[x][n] *= all;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                u32x4 wh[NV], wl[NV];
#pragma unroll
                for (int x = 0; x < NV; ++x)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const dc_f32x4 wk = *reinterpret_cast<const dc_f32x4 *>(scal + kScWk * 64 + 32 * s + 16 * i + 4 * g);
                        u32x2 hi, lo;
                        dc_split(X[x][2 * s + i] * wk, hi, lo);
                        wh[x][2 * i] = hi[0];
                        wh[x][2 * i + 1] = hi[1];
                        wl[x][2 * i] = lo[0];
                        wl[x][2 * i + 1] = lo[1];
                    }
#pragma unroll
                for (int n = 0; n < KT; ++n) {
                    const u32x4 kt = dc_ld_kt<D>(image, n, s, lane);
#pragma unroll
                    for (int x = 0; x < NV; ++x) {
                        S[x][n] = dc_mfma(kt, wl[x], S[x][n]);
                        S[x][n] = dc_mfma(kt, wh[x], S[x][n]);
                    }
                }
            }
        } else {
            if (more)
#pragma unroll
                for (int part = 1; part < 4; ++part)
                    fetch(ch + 1, part);
            // token by token, in the scaled units that the state has
            for (int t = 0; t < n_tok; ++t) {
                const float alpha = scal[kScAlpha * 64 + t], ks = scal[kScKs * 64 + t];
                const float beta = scal[kScBeta * 64 + t], qs = scal[kScQo * 64 + t];
#pragma unroll
                for (int x = 0; x < NV; ++x) {
                    const float vt = ld_elem<IO>(image + KQ + kDcHead + t * VP, (wave * NV + x) * 16 + c);
                    float sum = 0.0f;
                    dc_f32x4 k[KT];
#pragma unroll
                    for (int n = 0; n < KT; ++n) {
                        const u32x2 raw = *reinterpret_cast<const u32x2 *>(image + dc_at<D>(t, n, g));
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            k[n][r] = f16_to_f32(r % 2 ? raw[r / 2] >> 16 : raw[r / 2] & 0xffffu);
                            sum += S[x][n][r] * k[n][r];
                        }
                    }
                    sum = dc_sum_groups(sum);
                    const float u = beta * (vt * sc[x] - alpha * (sum * ks));
                    const float uk = u * ks;
#pragma unroll
                    for (int n = 0; n < KT; ++n)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            S[x][n][r] = S[x][n][r] * alpha + uk * k[n][r];
                    if (OUT) {
                        float o = 0.0f;
#pragma unroll
                        for (int n = 0; n < KT; ++n) {
                            const u32x2 raw = *reinterpret_cast<const u32x2 *>(image + KQ / 2 + dc_at<D>(t, n, g));
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                o += S[x][n][r] * f16_to_f32(r % 2 ? raw[r / 2] >> 16 : raw[r / 2] & 0xffffu);
                        }
                        o = dc_sum_groups(o) * qs / sc[x];
                        if (g == 0)
                            st_elem<IO>(p.out, b * p.out_bs + (tok0 + t) * p.out_ts + (int64_t)h * D + v0 + 16 * x + c, o);
                    }
                }
            }
            if (OUT)
                for (int t = n_tok; t < C && tok0 + t < p.seq_len; ++t)
                    if (g == 0)
#pragma unroll
                        for (int x = 0; x < NV; ++x)
                            st_elem<IO>(p.out, b * p.out_bs + (tok0 + t) * p.out_ts + (int64_t)h * D + v0 + 16 * x + c, 0.0f);
        }
    }

    if (w.last && !p.update)
        return;
#pragma unroll
    for (int x = 0; x < NV; ++x)
#pragma unroll
        for (int n = 0; n < KT; ++n) {
            const int o = (v0 + 16 * x + c) * D + 16 * n + 4 * g;
            const float f = 1.0f / sc[x];
            const float s[4] = {S[x][n][0] * f, S[x][n][1] * f, S[x][n][2] * f, S[x][n][3] * f};
            if (!w.last) {
                *reinterpret_cast<dc_f32x4 *>(carry + o) = dc_f32x4{s[0], s[1], s[2], s[3]};
            } else if (p.state_dtype == kF32) {
                delta_st_state(static_cast<float *>(p.state) + head_at + o, s);
            } else if (p.state_dtype == kF16) {
                delta_st_state(static_cast<_Float16 *>(p.state) + head_at + o, s);
            } else {
                delta_st_state(static_cast<bf16_t *>(p.state) + head_at + o, s);
            }
        }
}

template <typename IO, int D, int NV, int W>
hipError_t launch_delta_sweep(const DeltaParams &p, const DeltaWork &w, hipStream_t stream)
{
    const __int128 groups = (__int128)p.batch * p.hv * (D / (16 * W * NV));
    if (!launchable(groups, 64 * W))
        return hipErrorInvalidConfiguration;
    const uint32_t n = (uint32_t)groups;
    if (p.out)
        delta_sweep_kernel<IO, D, NV, W, true><<<dim3(n), 64 * W, 0, stream>>>(p, w, n % 8 == 0);
    else
        delta_sweep_kernel<IO, D, NV, W, false><<<dim3(n), 64 * W, 0, stream>>>(p, w, n % 8 == 0);
    return hipGetLastError();
}

template <typename IO, int D>
hipError_t launch_delta_chunks_d(const DeltaParams &p, const DeltaPlan &plan, hipStream_t stream)
{
    DeltaWork w = {};
    unsigned char *ws = static_cast<unsigned char *>(p.workspace);
    w.kq = ws;
    w.head = w.kq + plan.kq_bytes;
    w.carry = reinterpret_cast<float *>(w.head + plan.head_bytes);
    for (int c0 = 0; c0 < plan.chunks; c0 += plan.segment) {
        w.chunk0 = c0;
        w.chunks = min(plan.segment, plan.chunks - c0);
        w.first = c0 == 0;
        w.last = c0 + w.chunks >= plan.chunks;
        const __int128 groups = (__int128)w.chunks * p.hq * p.batch;
        if (!launchable(groups, 256) || p.batch > 65535)
            return hipErrorInvalidConfiguration;
        delta_prep_kernel<IO, D><<<dim3((uint32_t)(w.chunks * p.hq), p.batch), 256, 0, stream>>>(p, w);
        hipError_t e = hipGetLastError();
        if (e == hipSuccess)
            e = plan.wide ? launch_delta_sweep<IO, D, 1, D / 16>(p, w, stream)
                          : launch_delta_sweep<IO, D, 1, 4>(p, w, stream);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

template <typename IO>
hipError_t launch_delta_chunks_io(const DeltaParams &p, const DeltaPlan &plan, hipStream_t stream)
{
    return p.d == 64 ? launch_delta_chunks_d<IO, 64>(p, plan, stream)
                     : launch_delta_chunks_d<IO, 128>(p, plan, stream);
}

}  // namespace
}  // namespace ssu
