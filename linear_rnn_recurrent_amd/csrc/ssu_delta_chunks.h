// The gated delta rule in chunks of 64 or 32 tokens on the matrix cores.
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
// What bounds it: the chunks of a row follow each other, and in a workgroup of four waves each has
// a SIMD to itself, with nothing to hide its waits behind. 1 x 4096 tokens, 32 value heads of 128, bf16:
// prep 31 us (its waves wait 60 % of the time) and sweep 211, 3.3 a chunk; 106 MB are
// the least to move, 21 us. Rows fill the GPU with more waves: 8 x 4096 take 586 us, 1.5 TB/s.
//
// Precision: fp32 sums of products of fp16. k and q of 16 bits, scaled by a power of two to a
// length in [1, 2), are fp16 exactly but for what lies 2^-25 below that length; of fp32 they
// are pairs of fp16. L, P, the inverses, X, U and the state are pairs, hi + lo, 22 bits:
// their products keep fp32's accuracy to two bits, the state itself stays in fp32
// registers. For X, U and the state every value column has a power of two of its own,
// from z, twice the larger of max |v| and c max |S| of the column (|S k| <= c max |S|, c a
// little above the root of the number of keys): z in (2^5, 2^8]. With beta |k|^2 <= 1 a token
// only shrinks what is there and adds its v, so |U| <= 65 z < 2^15; up to 2.1 it grows by
// 1.1 at most, 64 of them by 2^9, and z stays in (2, 2^4]. What is cut off is 2^-25 of these
// units, 2^-30 of z. That is too much where strong decays leave nothing of a state, or of
// a v, that set the scale: with gamma_C < 2^-8 and a v of 16 tokens 2^-8 below z the chunk
// is not taken. A chunk with other values (without the norm; growing decays; a NaN or an
// infinity) is marked by prep, or seen by the wave, and runs token by token in the same
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
// deep; L, P and U go by pairs of tiles), or of one alone (16 deep, the inverses). S^T
// [key][value] is such an accumulator: it never leaves registers. K is kept with its
// keys in that order, in two planes of 8 bytes a lane, which both a row read (two
// planes) and a transposed read (ds_read_b64_tr_b16, one plane) take without bank conflicts.
#pragma once

#include "ssu_delta_impl.h"

namespace ssu {
namespace {

constexpr int kDcSpan = 64;       // tokens that a workgroup of prep takes: one chunk or two
constexpr int kDcTile = 1024;     // bytes of an inverse as [hi | lo], or of a plane (hi or lo) of two tiles

// Sizes by the type of the activations and the head: NT tiles of 16 tokens a chunk, PL fp16
// planes of k and q. Two chunks fit in LDS.
template <typename IO, int D>
struct DcShape {
    static constexpr int NT = delta_tiles(D, sizeof(IO) == 4), PL = sizeof(IO) == 4 ? 2 : 1;
    static constexpr int C = 16 * NT, CH = 4 / NT;  // tokens of a chunk, chunks of a span
    static constexpr int TILE = 32 * D;             // bytes of 16 tokens of k or q in a plane
    static constexpr int KQ = 2 * PL * NT * TILE;   // of K and Q of a chunk
    // Block of a value head and chunk: inverses, pairs of tiles of L (the second of rows 1
    // and 3's last is zero), scalars, pairs of P (what lies above the diagonal is zero)
    static constexpr int L = NT * kDcTile, SCALARS = L + (NT == 4 ? 4 : 1) * 2 * kDcTile;
    static constexpr int P = SCALARS + 8 * C * 4, HEAD = P + (NT == 4 ? 6 : 2) * 2 * kDcTile;
    static_assert(HEAD == delta_head_bytes(NT) && HEAD % 1024 == 0 && P % 1024 == 0, "block of a head");
    __device__ static constexpr int l_pair(int i, int p) { return L + (i - 1 + p) * 2 * kDcTile; }
    __device__ static constexpr int p_pair(int i, int p) { return P + (i < 2 ? i : 2 * i - 2 + p) * 2 * kDcTile; }
};
// Scalars: arrays of C floats
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
    unsigned char *kq;     // [batch][chunks][Hq]: K, then Q of a chunk, each in its planes
    unsigned char *head;   // [batch][chunks][HV][HEAD]
    float *carry;          // [batch][HV][D][D] between segments
    int chunk0, chunks;    // the segment: whole spans
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

// Four adjacent values, 8 or 16 bytes aligned, rounded to nearest even
template <typename IO>
__device__ __forceinline__ void dc_st4(IO *p, const float (&o)[4], bool live)
{
    if constexpr (sizeof(IO) == 4) {
        *reinterpret_cast<dc_f32x4 *>(p) = live ? dc_f32x4{o[0], o[1], o[2], o[3]} : dc_f32x4{0, 0, 0, 0};
    } else {
        u32x2 w;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const dc_f32x2 v = {o[2 * e], o[2 * e + 1]};
            if constexpr (__is_same(IO, _Float16))
                w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, dc_f16x2));
            else
                w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, dc_bf16x2));
        }
        *reinterpret_cast<u32x2 *>(p) = live ? w : u32x2{0, 0};
    }
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
    float beta[kDcSpan];   // beta_t k_s(t): of the fp16 keys
    float row[kDcSpan];    // decay from the tile's start through t
    float tail[kDcSpan];   // decay behind t to the tile's end, times k_s(t)
    float log[kDcSpan];
    float total[4];     // logs of a tile
};

template <typename IO, int D>
struct DcPrepLds {
    // planes of four tiles each
    unsigned char k[DcShape<IO, D>::PL][kDcSpan * D * 2], q[DcShape<IO, D>::PL][kDcSpan * D * 2];
    float ks[kDcSpan], qs[kDcSpan], kk[kDcSpan];  // length of k as fp16 -> k; of q -> scaled q; |k|^2
    float qq[kDcSpan];
    DcGates gates[4];
    float diag[4][16 * 20];
};

template <typename IO, int D>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaParams p, DeltaWork w)
{
    using Sh = DcShape<IO, D>;
    constexpr int KS = D / 32, NT = Sh::NT, PL = Sh::PL, C = Sh::C, CH = Sh::CH;
    __shared__ __attribute__((aligned(16))) DcPrepLds<IO, D> lds;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int G = p.hv / p.hq;
    const int span = blockIdx.x / p.hq, j = blockIdx.x - span * p.hq, b = blockIdx.y;
    const int pool = p.idx ? p.idx[b] : b;
    const int len = pool < 0 ? 0 : (p.ctx ? clamp_len(p.ctx[b], p.seq_len) : p.seq_len);
    const int t0 = w.chunk0 * C + span * kDcSpan;
    const int n = min(max(len - t0, 0), kDcSpan);
    if (p.out && (n + C - 1) / C < CH) {  // zeros in chunks behind the end, which sweep does not reach
        const int from = (n + C - 1) / C * C, to = min(p.seq_len - t0, kDcSpan), quads = G * D / 4;
        IO *o = static_cast<IO *>(p.out) + b * p.out_bs + (int64_t)j * G * D;
        const float zero[4] = {};
        for (int i = threadIdx.x; i < (to - from) * quads; i += 256) {
            const int t = i / quads;
            dc_st4<IO>(o + (t0 + from + t) * p.out_ts + 4 * (i - t * quads), zero, true);
        }
    }
    if (n == 0)
        return;

    // a and b of the first heads, a head a wave, lane = token: in flight with k and q
    float lg = 0.0f, beta = 0.0f;
    auto gates_of = [&](int head) {
        lg = beta = 0.0f;
        if (head < G && lane < n) {
            const int h = j * G + head;
            const int64_t t = t0 + lane;
            const float A = p.A_log ? -expf(p.A_log[h]) : 0.0f;
            const float bias = p.dt_bias ? ld_io(p.dt_bias, h, p.bias_dtype) : 0.0f;
            lg = delta_log_decay(p, A, bias, ld_io(p.a, b * p.a_bs + t * p.a_ts + h, p.gate_dtype));
            beta = delta_beta(p, ld_io(p.b, b * p.b_bs + t * p.b_ts + h, p.gate_dtype));
        }
    };

    // k and q of tile `wave`: lengths, fp16
    {
        const int tok = 16 * wave + c;
        const bool in = tok < n;
        const IO *kp = static_cast<const IO *>(p.k) + b * p.k_bs + (t0 + tok) * p.k_ts + j * D + 8 * g;
        const IO *qp = static_cast<const IO *>(p.q) + b * p.q_bs + (t0 + tok) * p.q_ts + j * D + 8 * g;
        u32x4 raw[2][KS][PL];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int x = 0; x < PL; ++x) {
                raw[0][ks][x] = raw[1][ks][x] = u32x4{0, 0, 0, 0};
                if (in) {
                    raw[0][ks][x] = reinterpret_cast<const u32x4 *>(kp + 32 * ks)[x];
                    if (p.out)
                        raw[1][ks][x] = reinterpret_cast<const u32x4 *>(qp + 32 * ks)[x];
                }
            }
        gates_of(wave);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float v[KS][8], sum = 0.0f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (PL == 2)
                        v[ks][e] = __uint_as_float(raw[s][ks][e / 4][e % 4]);
                    else
                        v[ks][e] = cvt_raw1<IO>(e % 2 ? raw[s][ks][0][e / 2] >> 16 : raw[s][ks][0][e / 2] & 0xffffu);
                    sum += v[ks][e] * v[ks][e];
                }
            sum = dc_sum_groups(sum);
            const bool fine = sum > 0.0f && sum < __builtin_inff();
            const int ex = fine ? min(max(1 - __builtin_amdgcn_frexp_expf(sqrtf(sum)), -126), 126) : 0;
            const float up = __builtin_amdgcn_ldexpf(1.0f, ex), down = __builtin_amdgcn_ldexpf(1.0f, -ex);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t h[PL][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = v[ks][2 * e] * up, y = v[ks][2 * e + 1] * up;
                    const dc_f16x2 hi = __builtin_convertvector((dc_f32x2){x, y}, dc_f16x2);
                    h[0][e] = __builtin_bit_cast(uint32_t, hi);
                    if constexpr (PL == 2)
                        h[1][e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(
                            (dc_f32x2){x - (float)hi[0], y - (float)hi[1]}, dc_f16x2));
                }
                // keys 32 ks + 8 g ..: pieces 2 g and 2 g + 1 of the eight pieces of a step
#pragma unroll
                for (int x = 0; x < PL; ++x) {
                    unsigned char *image = s ? lds.q[x] : lds.k[x];
                    *reinterpret_cast<u32x2 *>(image + dc_at<D>(tok, 2 * ks + (g >> 1), 2 * (g & 1))) = u32x2{h[x][0], h[x][1]};
                    *reinterpret_cast<u32x2 *>(image + dc_at<D>(tok, 2 * ks + (g >> 1), 2 * (g & 1) + 1)) = u32x2{h[x][2], h[x][3]};
                }
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
    const int64_t at = (int64_t)b * w.chunks + span * CH;
#pragma unroll
    for (int x = 0; x < PL; ++x)
#pragma unroll
        for (int i = 0; i < kDcSpan * D * 2 / 4096; ++i) {
            const int o = (i * 256 + threadIdx.x) * 16;
            const int sub = o / (NT * Sh::TILE), in = o - sub * (NT * Sh::TILE);
            unsigned char *to = w.kq + ((at + sub) * p.hq + j) * Sh::KQ + x * NT * Sh::TILE + in;
            *reinterpret_cast<u32x4 *>(to) = *reinterpret_cast<const u32x4 *>(lds.k[x] + o);
            if (p.out)
                *reinterpret_cast<u32x4 *>(to + Sh::KQ / 2) = *reinterpret_cast<const u32x4 *>(lds.q[x] + o);
        }

    // K_s . K_t and K_s . Q_t of the row tile `wave`: column t of the tile, rows s. L and P share
    // their decays, which weighs more than that the last tile's wave has the most columns.
    // i: the row tile within its chunk
    const int sub = wave / NT, i0 = sub * NT, i = wave - i0;
    dc_f32x4 kk[NT], qk[NT];
    auto dot = [&](const unsigned char *a0, const unsigned char *a1, int at, const unsigned char *b0,
                   const unsigned char *b1, int bt, dc_f32x4 x) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const u32x4 ah = dc_ld_op<D>(a0, at, ks, lane), bh = dc_ld_op<D>(b0, bt, ks, lane);
            if constexpr (PL == 2) {
                x = dc_mfma(dc_ld_op<D>(a1, at, ks, lane), bh, x);
                x = dc_mfma(ah, dc_ld_op<D>(b1, bt, ks, lane), x);
            }
            x = dc_mfma(ah, bh, x);
        }
        return x;
    };
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        kk[t] = qk[t] = dc_f32x4{0, 0, 0, 0};
        if (t <= i) {
            kk[t] = dot(lds.k[0], lds.k[PL - 1], i0 + t, lds.k[0], lds.k[PL - 1], i0 + i, kk[t]);
            if (p.out)
                qk[t] = dot(lds.k[0], lds.k[PL - 1], i0 + t, lds.q[0], lds.q[PL - 1], i0 + i, qk[t]);
        }
    }

    for (int h0 = 0; h0 < G; h0 += 4) {
        if (h0 + wave < G) {  // gates of four heads at once, lane = token
            const int h = j * G + h0 + wave;
            const bool in = lane < n;
            if (h0 > 0)
                gates_of(h0 + wave);
            const float ks = lds.ks[lane], qs = lds.qs[lane], kk2 = lds.kk[lane];
            const bool bad = in && !(lg <= 0.0f && kk2 <= 1.07f && fabsf(beta) * kk2 <= 2.1f &&
                                     (!p.out || lds.qq[lane] < __builtin_inff()));
            const bool wide = in && !(beta >= 0.0f && beta <= 1.02f && beta * kk2 <= 1.02f);
            const int mine = lane / C;  // chunk
            const uint64_t of_mine = (C == 64 ? ~(uint64_t)0 : (((uint64_t)1 << (C % 64)) - 1)) << (mine * C % 64);
            const float kind = __ballot(bad) & of_mine ? 1.0f : __ballot(wide) & of_mine ? 2.0f : 0.0f;
            const float row = row_prefix_sum16(lg);
            // behind the token to its tile's end: the suffix sum of the next token
            const float tail = dpp_f32_fill<0x101>(0.0f, row_suffix_sum16(lg));
            float total[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                total[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, row), 16 * i + 15));
            float before = 0.0f, behind = 0.0f, whole = 0.0f;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float part = x / NT == mine ? total[x] : 0.0f;
                before += x < g ? part : 0.0f;
                behind += x > g ? part : 0.0f;
                whole += part;
            }
            DcGates &s = lds.gates[wave];
            s.beta[lane] = beta * ks;
            s.row[lane] = expf(row);
            s.tail[lane] = expf(tail) * ks;
            s.log[lane] = lg;
            if (lane < 4)
                s.total[lane] = lane == 0 ? total[0] : lane == 1 ? total[1] : lane == 2 ? total[2] : total[3];
            float *sc = reinterpret_cast<float *>(w.head + ((at + mine) * p.hv + h) * Sh::HEAD + Sh::SCALARS) + lane % C;
            const float gamma = expf(before + row);
            sc[kScBeta * C] = beta;
            sc[kScGk * C] = gamma * ks;
            sc[kScWk * C] = expf(behind + tail) * ks;
            sc[kScAlpha * C] = expf(lg);
            sc[kScKs * C] = ks;
            sc[kScGo * C] = gamma * qs;
            sc[kScQo * C] = qs;
            sc[kScMisc * C] = lane % C == 0 ? expf(whole) : lane % C == 1 ? kind : 0.0f;
        }
        __syncthreads();
        for (int hh = 0; hh < 4 && h0 + hh < G; ++hh) {
            const DcGates &s = lds.gates[hh];
            unsigned char *to = w.head + ((at + sub) * p.hv + j * G + h0 + hh) * Sh::HEAD;
            const int t = 16 * (i0 + i) + c;
            const float own = s.beta[t], row = s.row[t];
            // a tile of L (with its sign in U's recursion) and one of P from their common factors
            auto put = [&](unsigned char *at8, const dc_f32x4 &v) {
                u32x2 hi, lo;
                dc_split(v, hi, lo);
                *reinterpret_cast<u32x2 *>(at8) = hi;
                *reinterpret_cast<u32x2 *>(at8 + kDcTile) = lo;
            };
#pragma unroll
            for (int jt = 0; jt < NT - 1; ++jt) {
                if (jt >= i)
                    break;
                float mid = 0.0f;
                for (int m = jt + 1; m < i; ++m)
                    mid += s.total[i0 + m];
                const float f = row * expf(mid);
                const dc_f32x4 tail = *reinterpret_cast<const dc_f32x4 *>(&s.tail[16 * (i0 + jt) + 4 * g]) * f;
                put(to + Sh::l_pair(i, jt >> 1) + lane * 16 + 8 * (jt & 1), tail * kk[jt] * -own);
                if (p.out)
                    put(to + Sh::p_pair(i, jt >> 1) + lane * 16 + 8 * (jt & 1), tail * qk[jt]);
            }
            // diagonal tile: decays behind s through t by adding from t downwards
            float logs[16];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const dc_f32x4 x = *reinterpret_cast<const dc_f32x4 *>(&s.log[16 * (i0 + i) + 4 * q]);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    logs[4 * q + r] = x[r];
            }
            float sum = 0.0f;
            dc_f32x4 dl = {0, 0, 0, 0};
#pragma unroll
            for (int m = 15; m >= 1; --m) {
                sum += m <= c ? logs[m] : 0.0f;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if ((m - 1) % 4 == r)
                        dl[r] = g == (m - 1) / 4 ? sum : dl[r];
            }
            const dc_f32x4 ks = *reinterpret_cast<const dc_f32x4 *>(&lds.ks[16 * (i0 + i) + 4 * g]);
            dc_f32x4 x = kk[NT - 1], y = qk[NT - 1];
#pragma unroll
            for (int q = 0; q < NT - 1; ++q)
                if (i == q) {
                    x = kk[q];
                    y = qk[q];
                }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float d = expf(dl[r]) * ks[r];
                x[r] = 4 * g + r < c ? d * own * x[r] : 0.0f;
                y[r] = 4 * g + r <= c ? d * y[r] : 0.0f;
            }
            if (p.out) {
                unsigned char *at8 = to + Sh::p_pair(i, i >> 1) + lane * 16 + 8 * (i & 1);
                put(at8, y);
                if (!(i & 1))
                    *reinterpret_cast<u32x2 *>(at8 + 8) = *reinterpret_cast<u32x2 *>(at8 + kDcTile + 8) = u32x2{0, 0};
            }
            float *tile = lds.diag[wave];
            __builtin_amdgcn_wave_barrier();
            *reinterpret_cast<dc_f32x4 *>(tile + c * 20 + 4 * g) = x;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            float L[16];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const dc_f32x4 z = *reinterpret_cast<const dc_f32x4 *>(tile + c * 20 + 4 * q);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    L[4 * q + r] = z[r];
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int r = 0; r < 4; ++r)
                x[r] = 4 * g + r == c ? 1.0f : 0.0f;
            dc_invert<0>(L, x);
            u32x2 hi, lo;
            dc_split(x, hi, lo);
            *reinterpret_cast<u32x4 *>(to + i * kDcTile + lane * 16) = u32x4{hi[0], hi[1], lo[0], lo[1]};
            if (i & 1) {  // the second tile of this row's last pair
                unsigned char *at8 = to + Sh::l_pair(i, i >> 1) + lane * 16 + 8;
                *reinterpret_cast<u32x2 *>(at8) = *reinterpret_cast<u32x2 *>(at8 + kDcTile) = u32x2{0, 0};
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

// Values of four tokens 4 g + r of tile i, column c of the wave's, from token rows in LDS
template <typename IO, int PITCH>
struct DcValues {
    u32x2 w;

    __device__ __forceinline__ void load(unsigned char *rows, int i, int lane)
    {
        const int g = lane >> 4, x = lane & 15;
        unsigned char *p = rows + (16 * i + 4 * g + (x >> 2)) * PITCH + (x & 3) * 8;
        w = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((dc_lds_v4)p));
    }
    __device__ __forceinline__ void keep(int n)  // the first n of the four
    {
        w[0] &= (n > 0 ? 0xffffu : 0u) | (n > 1 ? 0xffff0000u : 0u);
        w[1] &= (n > 2 ? 0xffffu : 0u) | (n > 3 ? 0xffff0000u : 0u);
    }
    __device__ __forceinline__ float operator[](int r) const
    {
        return cvt_raw1<IO>(r % 2 ? w[r / 2] >> 16 : w[r / 2] & 0xffffu);
    }
    // bits of the largest magnitude as fp32; those of a NaN above infinity's
    __device__ __forceinline__ uint32_t most() const
    {
        const uint32_t m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(
            __builtin_bit_cast(dc_u16x2, w[0] & 0x7fff7fffu), __builtin_bit_cast(dc_u16x2, w[1] & 0x7fff7fffu)));
        return __float_as_uint(cvt_raw1<IO>(max(m & 0xffffu, m >> 16)));
    }
};

template <int PITCH>
struct DcValues<float, PITCH> {
    uint32_t w[4];

    __device__ __forceinline__ void load(unsigned char *rows, int i, int lane)
    {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            w[r] = *reinterpret_cast<const uint32_t *>(rows + (16 * i + 4 * (lane >> 4) + r) * PITCH + (lane & 15) * 4);
    }
    __device__ __forceinline__ void keep(int n)
    {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            w[r] = r < n ? w[r] : 0;
    }
    __device__ __forceinline__ float operator[](int r) const { return __uint_as_float(w[r]); }
    __device__ __forceinline__ uint32_t most() const
    {
        return max(max(w[0] & 0x7fffffffu, w[1] & 0x7fffffffu), max(w[2] & 0x7fffffffu, w[3] & 0x7fffffffu));
    }
};

// One wave: 16 value columns of value head h, batch entry b.
template <typename IO, int D, int W, bool OUT>
__global__ __launch_bounds__(64 * W, W > 4 ? 2 : 1) void delta_sweep_kernel(DeltaParams p, DeltaWork w, int swizzle)
{
    using Sh = DcShape<IO, D>;
    constexpr int KS = D / 32, KT = D / 16, NT = Sh::NT, PL = Sh::PL, C = Sh::C, NP = NT / 2;
    constexpr int TILES = D / (16 * W);                // workgroups a head
    constexpr int KQ = Sh::KQ, VP = 16 * W * sizeof(IO);  // bytes of K and Q, of a token's values
    constexpr int BUF = KQ + Sh::HEAD + C * VP;        // of a chunk in LDS
    constexpr int PLANE = NT * Sh::TILE;
    static_assert(TILES * 16 * W == D && 2 * BUF <= 160 * 1024, "value columns of a head; LDS");
    __shared__ __attribute__((aligned(16))) unsigned char lds[2 * BUF];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    // workgroups are dealt out over eight XCDs: those of one q head go to the same one
    const uint32_t id = swizzle ? (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3) : blockIdx.x;
    const int64_t bh = id / TILES;
    const int b = (int)(bh / p.hv), h = (int)(bh - (int64_t)b * p.hv);
    const int wg_v0 = (int)(id - bh * TILES) * (16 * W), v0 = wg_v0 + wave * 16;
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
    const unsigned char *hd = w.head + ((int64_t)b * w.chunks * p.hv + h) * Sh::HEAD + lane * 16;
    const int64_t kq_step = (int64_t)p.hq * KQ, hd_step = (int64_t)p.hv * Sh::HEAD;
    constexpr int VL = VP / 16, VR = 64 / VL;  // lanes a token's values, tokens an instruction
    static_assert(C % (VR * W) == 0, "the same number of value loads for every wave");
    const IO *vp = static_cast<const IO *>(p.v) + b * p.v_bs + (int64_t)w.chunk0 * C * p.v_ts +
                   (int64_t)h * D + wg_v0 + 16 / sizeof(IO) * (lane % VL);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char *)lds;
    // part 0 .. 3 of four (the CU takes 64 bytes a cycle: issued at once, they would stall the wave)
    auto fetch = [&](int ch, int part) {
        uint32_t to = lds0 + (ch & 1) * BUF;
        const unsigned char *from = kq + ch * kq_step;
        constexpr int QK = OUT ? KQ : KQ / 2;
        static_assert(QK % (W * 1024) == 0, "the same number of loads for every wave");
#pragma unroll
        for (int o = 0; o < QK; o += W * 1024)
            if (o / (W * 1024) % 4 == part)
                dc_to_lds(from + o + wave * 1024, to + o + wave * 1024);
        to += KQ;
        from = hd + ch * hd_step;
        constexpr int HD = OUT ? Sh::HEAD : Sh::P;
#pragma unroll
        for (int o = 0; o < HD; o += W * 1024)
            if (o / (W * 1024) % 4 == part && (o + W * 1024 <= HD || o + wave * 1024 < HD))
                dc_to_lds(from + o + wave * 1024, to + o + wave * 1024);
        to += Sh::HEAD;
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
    dc_f32x4 S[KT];
    const int64_t head_at = pool * p.row_stride + (int64_t)h * D * D;
    float *carry = w.carry + ((int64_t)b * p.hv + h) * D * D;
    if (!w.first || p.state_dtype == kF32) {
        const float *s = (w.first ? static_cast<const float *>(p.state) + head_at : carry) + (v0 + c) * D + 4 * g;
#pragma unroll
            for (int n = 0; n < KT; ++n)
                S[n] = *reinterpret_cast<const dc_f32x4 *>(s + 16 * n);
    } else {
        const uint16_t *s = static_cast<const uint16_t *>(p.state) + head_at + (v0 + c) * D + 4 * g;
        u32x2 raw[KT];
#pragma unroll
            for (int n = 0; n < KT; ++n)
                raw[n] = *reinterpret_cast<const u32x2 *>(s + 16 * n);
        auto widen = [&](auto tag) {
#pragma unroll
                for (int n = 0; n < KT; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        S[n][r] = cvt_raw1<decltype(tag)>(r % 2 ? raw[n][r / 2] >> 16 : raw[n][r / 2] & 0xffffu);
        };
        if (p.state_dtype == kF16)
            widen(_Float16{});
        else
            widen(bf16_t{});
    }
    IO *op = static_cast<IO *>(p.out) + b * p.out_bs + (int64_t)h * D + v0;
    const int o_off = c * (int)p.out_ts + 4 * g;
    float sc = 1.0f;                         // scale of the value column of this lane
    float isc[4] = {1.0f, 1.0f, 1.0f, 1.0f};  // 1 / scale of value columns 4 g + r
    // |S k| <= bound max |S|
    constexpr float kBound = D == 32 ? 6.0f : D == 64 ? 8.5f : D == 128 ? 12.0f : 16.5f;

    for (int ch = 0; ch < chunks; ++ch) {
        // this chunk's LDS is filled (by every wave: behind the barrier), the other one read
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        unsigned char *image = lds + (ch & 1) * BUF;
        const unsigned char *blk = image + KQ;
        const float *scal = reinterpret_cast<const float *>(blk + Sh::SCALARS);
        const int t0 = ch * C, n_tok = min(mine - t0, C);
        const int64_t tok0 = (int64_t)w.chunk0 * C + t0;
        const bool more = ch + 1 < chunks;
        if (more)
            fetch(ch + 1, 0);
        DcValues<IO, VP> v[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i)
            v[i].load(image + KQ + Sh::HEAD + wave * 16 * (int)sizeof(IO), i, lane);
        if (n_tok < C) {  // what was read in the place of tokens behind the end
#pragma unroll
            for (int i = 0; i < NT; ++i)
                v[i].keep(n_tok - (16 * i + 4 * g));
        }

        u32x4 kf[PL][NT];  // in flight over the scales
#pragma unroll
        for (int x = 0; x < PL; ++x)
#pragma unroll
            for (int i = 0; i < NT; ++i)
                kf[x][i] = dc_ld_op<D>(image + x * PLANE, i, 0, lane);

        // scales, and whether the chunk may run on the matrix cores
        const float all = scal[kScMisc * C], kind = scal[kScMisc * C + 1];
        const float top = kind == 2.0f ? 0x1p4f : 0x1p8f;
        const bool fades = all < 0x1p-8f;
        bool slow = kind == 1.0f;
        float ms[2] = {0.0f, 0.0f};  // a NaN of the state reaches every token of the chunk anyway
#pragma unroll
        for (int n = 0; n < KT; ++n)
            ms[n & 1] = fmaxf(fmaxf(fmaxf(ms[n & 1], fabsf(S[n][0])), fabsf(S[n][1])),
                              fmaxf(fabsf(S[n][2]), fabsf(S[n][3])));
        uint32_t tile[NT], mv = 0;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            tile[i] = v[i].most();
            mv = max(mv, tile[i]);
        }
        slow |= mv >= 0x7f800000u;
        // z from one exchange: twice the larger of its two parts
        const float part = fmaxf(__uint_as_float(mv) * sc, kBound * fmaxf(ms[0], ms[1]));
        const float z = 2.0f * __uint_as_float(dc_max_groups(__float_as_uint(part)));
        slow |= !(z < __builtin_inff());
        if (fades) {
            uint32_t least = 0x7f800000u;  // of whole tiles
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint32_t m = dc_max_groups(tile[i]);
                least = n_tok >= 16 * i + 16 ? min(least, m) : least;
            }
            slow |= __uint_as_float(least) * sc < z * 0x1p-8f;
        }
        const bool move = z > top || (z <= top * 0x1p-3f && z > 0.0f);
        slow = __ballot(slow) != 0;
        if (!slow && __ballot(move)) {
            int k = move ? __builtin_amdgcn_frexp_expf(top) - 1 - __builtin_amdgcn_frexp_expf(z) : 0;
            // the scale itself stays within 2^-124 .. 2^124, which every finite z reaches
            const int e = __builtin_amdgcn_frexp_expf(sc) - 1;
            k = min(max(k, -124 - e), 124 - e);
            const float f = __builtin_amdgcn_ldexpf(1.0f, k);
            sc *= f;
#pragma unroll
            for (int n = 0; n < KT; ++n)
                S[n] *= f;
            const float inv = __builtin_amdgcn_ldexpf(1.0f, -(e + k));
#pragma unroll
            for (int r = 0; r < 4; ++r)
                isc[r] = __shfl(inv, 4 * g + r, 64);
        }

        if (!slow) {
            dc_f32x4 X[NT], O[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i)
                X[i] = O[i] = dc_f32x4{0, 0, 0, 0};
            // S0 k and S0 q
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                u32x2 h0, l0, h1, l1;
                dc_split(S[2 * ks], h0, l0);
                dc_split(S[2 * ks + 1], h1, l1);
                const u32x4 sh = {h0[0], h0[1], h1[0], h1[1]}, sl = {l0[0], l0[1], l1[0], l1[1]};
                u32x4 qf[PL][NT], kn[PL][NT];
#pragma unroll
                for (int x = 0; x < PL; ++x)
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        if (OUT)
                            qf[x][i] = dc_ld_op<D>(image + KQ / 2 + x * PLANE, i, ks, lane);
                        if (ks + 1 < KS)
                            kn[x][i] = dc_ld_op<D>(image + x * PLANE, i, ks + 1, lane);
                    }
#pragma unroll
                for (int x = 0; x < PL; ++x)
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        X[i] = dc_mfma(kf[x][i], sh, X[i]);
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    X[i] = dc_mfma(kf[0][i], sl, X[i]);
                if (OUT) {
#pragma unroll
                    for (int x = 0; x < PL; ++x)
#pragma unroll
                        for (int i = 0; i < NT; ++i)
                            O[i] = dc_mfma(sh, qf[x][i], O[i]);
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        O[i] = dc_mfma(sl, qf[0][i], O[i]);
                }
                if (ks + 1 < KS)
#pragma unroll
                    for (int x = 0; x < PL; ++x)
#pragma unroll
                        for (int i = 0; i < NT; ++i)
                            kf[x][i] = kn[x][i];
            }
            if (more)
                fetch(ch + 1, 1);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const dc_f32x4 beta = *reinterpret_cast<const dc_f32x4 *>(scal + kScBeta * C + 16 * i + 4 * g);
                const dc_f32x4 gk = *reinterpret_cast<const dc_f32x4 *>(scal + kScGk * C + 16 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    X[i][r] = beta[r] * (v[i][r] * sc - gk[r] * X[i][r]);
            }
            if (more)
                fetch(ch + 1, 2);
            // U, tile after tile: 32-deep operands are pairs of tiles
            u32x4 uh[NP], ul[NP];
#pragma unroll
            for (int q = 0; q < NP; ++q)
                uh[q] = ul[q] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < NT; ++i) {
#pragma unroll
                for (int q = 0; 2 * q < i; ++q) {
                    const u32x4 lh = *reinterpret_cast<const u32x4 *>(blk + Sh::l_pair(i, q) + lane * 16);
                    const u32x4 ll = *reinterpret_cast<const u32x4 *>(blk + Sh::l_pair(i, q) + kDcTile + lane * 16);
                    X[i] = dc_mfma(ll, uh[q], X[i]);
                    X[i] = dc_mfma(lh, ul[q], X[i]);
                    X[i] = dc_mfma(lh, uh[q], X[i]);
                }
                const u32x4 df = *reinterpret_cast<const u32x4 *>(blk + i * kDcTile + lane * 16);
                const u32x2 dh = {df[0], df[1]}, dl = {df[2], df[3]};
                u32x2 hi, lo;
                dc_split(X[i], hi, lo);
                dc_f32x4 u = {0, 0, 0, 0};
                u = dc_mfma16(dl, hi, u);
                u = dc_mfma16(dh, lo, u);
                u = dc_mfma16(dh, hi, u);
                X[i] = u;
                dc_split(u, hi, lo);
                uh[i >> 1][2 * (i & 1)] = hi[0];
                uh[i >> 1][2 * (i & 1) + 1] = hi[1];
                ul[i >> 1][2 * (i & 1)] = lo[0];
                ul[i >> 1][2 * (i & 1) + 1] = lo[1];
            }
            if (more)
                fetch(ch + 1, 3);
            if (OUT) {
                dc_f32x4 Q[NT];
#pragma unroll
                for (int r = 0; r < NP; ++r)
#pragma unroll
                    for (int i = 2 * r; i < NT; ++i) {
                        const u32x4 ph = *reinterpret_cast<const u32x4 *>(blk + Sh::p_pair(i, r) + lane * 16);
                        const u32x4 pl = *reinterpret_cast<const u32x4 *>(blk + Sh::p_pair(i, r) + kDcTile + lane * 16);
                        if (r == 0)
                            Q[i] = dc_f32x4{0, 0, 0, 0};
                        Q[i] = dc_mfma(uh[r], pl, Q[i]);
                        Q[i] = dc_mfma(ul[r], ph, Q[i]);
                        Q[i] = dc_mfma(uh[r], ph, Q[i]);
                    }
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const float go = scal[kScGo * C + 16 * i + c], qo = scal[kScQo * C + 16 * i + c];
                    float o[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        o[r] = isc[r] * (go * O[i][r] + qo * Q[i][r]);
                    IO *to = op + (tok0 + 16 * i) * p.out_ts + o_off;
                    if (n_tok == C)
                        dc_st4<IO>(to, o, true);
                    else if (tok0 + 16 * i + c < p.seq_len)
                        dc_st4<IO>(to, o, 16 * i + c < n_tok);
                }
            }
            // the state behind the chunk
#pragma unroll
            for (int n = 0; n < KT; ++n)
                S[n] *= all;
#pragma unroll
            for (int s = 0; s < NP; ++s) {
                u32x4 wh, wl;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const dc_f32x4 wk = *reinterpret_cast<const dc_f32x4 *>(scal + kScWk * C + 32 * s + 16 * i + 4 * g);
                    u32x2 hi, lo;
                    dc_split(X[2 * s + i] * wk, hi, lo);
                    wh[2 * i] = hi[0];
                    wh[2 * i + 1] = hi[1];
                    wl[2 * i] = lo[0];
                    wl[2 * i + 1] = lo[1];
                }
#pragma unroll
                for (int n = 0; n < KT; ++n) {
                    const u32x4 kt = dc_ld_kt<D>(image, n, s, lane);
                    if constexpr (PL == 2)
                        S[n] = dc_mfma(dc_ld_kt<D>(image + PLANE, n, s, lane), wh, S[n]);
                    S[n] = dc_mfma(kt, wl, S[n]);
                    S[n] = dc_mfma(kt, wh, S[n]);
                }
            }
        } else {
            if (more)
#pragma unroll
                for (int part = 1; part < 4; ++part)
                    fetch(ch + 1, part);
            // token by token, in the scaled units that the state has
            auto ld_keys = [&](const unsigned char *at, int t, int n) {
                dc_f32x4 k;
#pragma unroll
                for (int x = 0; x < PL; ++x) {
                    const u32x2 bits = *reinterpret_cast<const u32x2 *>(at + x * PLANE + dc_at<D>(t, n, g));
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float f = f16_to_f32(r % 2 ? bits[r / 2] >> 16 : bits[r / 2] & 0xffffu);
                        k[r] = x ? k[r] + f : f;
                    }
                }
                return k;
            };
            for (int t = 0; t < n_tok; ++t) {
                const float alpha = scal[kScAlpha * C + t], ks = scal[kScKs * C + t];
                const float beta = scal[kScBeta * C + t], qs = scal[kScQo * C + t];
                const float vt = ld_elem<IO>(image + KQ + Sh::HEAD + t * VP, wave * 16 + c);
                float sum = 0.0f;
                for (int n = 0; n < KT; ++n) {
                    const dc_f32x4 k = ld_keys(image, t, n);
#pragma unroll
                    for (int m = 0; m < KT; ++m)
                        if (m == n)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                sum += S[m][r] * k[r];
                }
                sum = dc_sum_groups(sum);
                const float u = beta * (vt * sc - alpha * (sum * ks));
                const float uk = u * ks;
                float o = 0.0f;
                for (int n = 0; n < KT; ++n) {
                    const dc_f32x4 k = ld_keys(image, t, n);
                    dc_f32x4 q = {0, 0, 0, 0};
                    if (OUT)
                        q = ld_keys(image + KQ / 2, t, n);
#pragma unroll
                    for (int m = 0; m < KT; ++m)
                        if (m == n)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                S[m][r] = S[m][r] * alpha + uk * k[r];
                                o += S[m][r] * q[r];
                            }
                }
                if (OUT) {
                    o = dc_sum_groups(o) * qs / sc;
                    if (g == 0)
                        st_elem<IO>(op + (tok0 + t) * p.out_ts, c, o);
                }
            }
            if (OUT && g == 0)
                for (int t = n_tok; t < C && tok0 + t < p.seq_len; ++t)
                    st_elem<IO>(op + (tok0 + t) * p.out_ts, c, 0.0f);
        }
    }

    if (w.last && !p.update)
        return;
    const float f = 1.0f / sc;
#pragma unroll
    for (int n = 0; n < KT; ++n) {
        const int o = (v0 + c) * D + 16 * n + 4 * g;
        const float s[4] = {S[n][0] * f, S[n][1] * f, S[n][2] * f, S[n][3] * f};
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

template <typename IO, int D, int W>
hipError_t launch_delta_sweep(const DeltaParams &p, const DeltaWork &w, hipStream_t stream)
{
    const __int128 groups = (__int128)p.batch * p.hv * (D / (16 * W));
    if (!launchable(groups, 64 * W))
        return hipErrorInvalidConfiguration;
    const uint32_t n = (uint32_t)groups;
    if (p.out)
        delta_sweep_kernel<IO, D, W, true><<<dim3(n), 64 * W, 0, stream>>>(p, w, n % 8 == 0);
    else
        delta_sweep_kernel<IO, D, W, false><<<dim3(n), 64 * W, 0, stream>>>(p, w, n % 8 == 0);
    return hipGetLastError();
}

template <typename IO, int D>
hipError_t launch_delta_chunks_d(const DeltaParams &p, const DeltaPlan &plan, hipStream_t stream)
{
    using Sh = DcShape<IO, D>;
    // fp32 rows of 256 leave room for the values of two waves
    constexpr int W = D == 32 || (D == 256 && sizeof(IO) == 4) ? 2 : 4, WIDE = D >= 128 && W == 4 ? 8 : W;
    DeltaWork w = {};
    unsigned char *ws = static_cast<unsigned char *>(p.workspace);
    w.kq = ws;
    w.head = w.kq + plan.kq_bytes;
    w.carry = reinterpret_cast<float *>(w.head + plan.head_bytes);
    for (int s0 = 0; s0 < plan.spans; s0 += plan.segment) {
        const int spans = min(plan.segment, plan.spans - s0);
        w.chunk0 = s0 * Sh::CH;
        w.chunks = spans * Sh::CH;
        w.first = s0 == 0;
        w.last = s0 + spans >= plan.spans;
        if (!launchable((__int128)spans * p.hq * p.batch, 256) || p.batch > 65535)
            return hipErrorInvalidConfiguration;
        delta_prep_kernel<IO, D><<<dim3((uint32_t)(spans * p.hq), p.batch), 256, 0, stream>>>(p, w);
        hipError_t e = hipGetLastError();
        if (e == hipSuccess)
            e = plan.wide ? launch_delta_sweep<IO, D, WIDE>(p, w, stream)
                          : launch_delta_sweep<IO, D, W>(p, w, stream);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

template <typename IO>
hipError_t launch_delta_chunks_io(const DeltaParams &p, const DeltaPlan &plan, hipStream_t stream)
{
    switch (p.d) {
    case 32: return launch_delta_chunks_d<IO, 32>(p, plan, stream);
    case 64: return launch_delta_chunks_d<IO, 64>(p, plan, stream);
    case 128: return launch_delta_chunks_d<IO, 128>(p, plan, stream);
    default: return launch_delta_chunks_d<IO, 256>(p, plan, stream);
    }
}

}  // namespace
}  // namespace ssu
