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
// tile after tile (U_i = (I + L_ii)^-1 X_i, then X_j -= L_ji U_i for the tiles j behind it).
//
// What bounds it: the chunks of a row follow each other, and in a workgroup of four waves (and a fifth that
// fetches) each has a SIMD to itself, with nothing to hide its waits behind. 1 x 4096 tokens, 32 value heads of
// 128, bf16: prep 33 us and sweep 245, 3.8 a chunk, of which 204 matrix instructions keep their unit busy for
// 1.4 and 850 vector instructions theirs; 106 MB are the least to move, 21 us. Rows fill the GPU with more
// waves: 8 x 4096 take 690 us.
//
// Precision: fp32 sums of products of bf16, which has fp32's range. What is of fp32 (the state, L, P,
// the inverses, X, U; k and q of that type) goes into them as three parts, hi + mid + lo, 24 bits of every
// entry for itself, whatever stands beside it; k and q of fp16 are two parts, of bf16 one. Six of the
// nine products of two triples are formed; those left out are 2^-24 of it. So a chunk is as near to the
// formula as the recurrence in fp32, but where rounding errors grow: with beta (k . k) of 2.02 and the same key
// in 512 tokens they are 2e-4 of the outputs, the recurrence's 3e-6 (with 2, 3e-5 and 5e-6), and betas outside
// [-1, 2] / (k . k), but for their rounding, are not taken. Pairs of fp16 do with 138 matrix instructions, but cover 25 bits below a unit that a column shares: what is
// small beside its largest value, of whichever token, loses digits.
// A chunk that prep marks (such betas; growing decays, whose sums of logarithms cancel; a NaN or an
// infinity in k or a gate), or whose U turns out not finite, runs token by token in the same
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
// deep), or two parts of one (the inverses, L and P: a product of 16 slots has two products of parts in
// an instruction). S^T [key][value] is such an accumulator: it never leaves registers. K is kept with its
// keys in that order, in two halves of 8 bytes a lane, which both a row read (two
// halves) and a transposed read (ds_read_b64_tr_b16, one half) take without bank conflicts.
#pragma once

#include "ssu_delta_impl.h"

namespace ssu {
namespace {

constexpr int kDcSpan = 64;       // tokens that a workgroup of prep takes: one chunk or two
constexpr int kDcTile = 1536;     // bytes of 16 x 16 entries in three parts: [hi | mid] by lanes, then lo

// Sizes by the type of the activations and the head: NT tiles of 16 tokens a chunk, PL planes (parts)
// of k and q. Two chunks fit in LDS, but of fp32 heads of 256.
template <typename IO, int D>
struct DcShape {
    static constexpr int PL = delta_planes(sizeof(IO) == 4 ? kF32 : __is_same(IO, _Float16) ? kF16 : kBF16);
    static constexpr int NT = delta_tiles(D, PL);
    static constexpr int C = 16 * NT, CH = 4 / NT;  // tokens of a chunk, chunks of a span
    static constexpr int TILE = 32 * D;             // bytes of 16 tokens of k or q in a plane
    static constexpr int KQ = 2 * PL * NT * TILE;   // of K and Q of a chunk
    // Block of a value head and chunk, in tiles: inverses, L below the diagonal, scalars, P up to it
    static constexpr int L = NT * kDcTile, SCALARS = L + NT * (NT - 1) / 2 * kDcTile;
    static constexpr int P = SCALARS + 8 * C * 4, HEAD = P + NT * (NT + 1) / 2 * kDcTile;
    static_assert(HEAD == delta_head_bytes(NT) && HEAD % 1024 == 0, "block of a head");
    static constexpr int buffer(int waves) { return KQ + HEAD + waves * C * 16 * (int)sizeof(IO); }
    static constexpr int buffers(int waves) { return 2 * buffer(waves) <= 160 * 1024 ? 2 : 1; }
    __device__ static constexpr int l_tile(int i, int s) { return L + (i * (i - 1) / 2 + s) * kDcTile; }
    __device__ static constexpr int p_tile(int i, int s) { return P + (i * (i + 1) / 2 + s) * kDcTile; }
};
// Scalars: arrays of C floats
enum : int { kScBeta, kScGk, kScWk, kScAlpha, kScKs, kScGo, kScQo, kScMisc };

typedef _Float16 dc_f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 dc_bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 dc_bf16x8 __attribute__((ext_vector_type(8)));
typedef float dc_f32x2 __attribute__((ext_vector_type(2)));
typedef float dc_f32x4 __attribute__((ext_vector_type(4)));
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
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(dc_bf16x8, a),
                                                   __builtin_bit_cast(dc_bf16x8, b), c, 0, 0, 0);
}

// Which of the products of PA and PB parts are formed, the smallest first: not those of 2^-24 of the whole of
// two triples, nor lo lo' of a pair and a triple (an fp16's second part has three bits). f(i, j)
template <int PA, int PB, typename F>
__device__ __forceinline__ void dc_each(F f)
{
#pragma unroll
    for (int order = PA + PB - 2 < 2 ? PA + PB - 2 : 2; order >= 0; --order)
#pragma unroll
        for (int i = 0; i < PA; ++i)
            if (order - i >= 0 && order - i < PB)
                f(i, order - i);
}

// Two adjacent fp32 as a pair of bf16, and what that leaves (exact)
__device__ __forceinline__ uint32_t dc_part(float &a, float &b)
{
    const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector((dc_f32x2){a, b}, dc_bf16x2));
    a -= __uint_as_float(w << 16);
    b -= __uint_as_float(w & 0xffff0000u);
    return w;
}

// Four fp32 values as three parts. Two roundings to nearest leave seven bits at most: the third
// part is exact.
__device__ __forceinline__ void dc_split(const dc_f32x4 &f, u32x2 (&part)[3])
{
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float a = f[2 * e], b = f[2 * e + 1];
        part[0][e] = dc_part(a, b);
        part[1][e] = dc_part(a, b);
        part[2][e] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
    }
}

// Two of them as an operand of 32 slots
__device__ __forceinline__ void dc_split2(const dc_f32x4 &f, const dc_f32x4 &g, u32x4 (&op)[3])
{
    u32x2 a[3], b[3];
    dc_split(f, a);
    dc_split(g, b);
#pragma unroll
    for (int x = 0; x < 3; ++x)
        op[x] = u32x4{a[x][0], a[x][1], b[x][0], b[x][1]};
}

// A product of 16 slots takes two parts of either side in one instruction. Of a tile in memory: [hi | mid] and
// [hi | lo], against [lo | hi], [mid | hi] and [hi | mid] of the other.
struct DcTile {
    u32x4 hm, hl;

    __device__ __forceinline__ void load(const unsigned char *at, int lane)
    {
        hm = *reinterpret_cast<const u32x4 *>(at + lane * 16);
        const u32x2 lo = *reinterpret_cast<const u32x2 *>(at + 1024 + lane * 8);
        hl = u32x4{hm[0], hm[1], lo[0], lo[1]};
    }
};
__device__ __forceinline__ void dc_st_tile(unsigned char *at, int lane, const dc_f32x4 &f)
{
    u32x2 x[3];
    dc_split(f, x);
    *reinterpret_cast<u32x4 *>(at + lane * 16) = u32x4{x[0][0], x[0][1], x[1][0], x[1][1]};
    *reinterpret_cast<u32x2 *>(at + 1024 + lane * 8) = x[2];
}
struct DcOther {
    u32x4 lh, mh, hm;

    __device__ __forceinline__ explicit DcOther(const dc_f32x4 &f)
    {
        u32x2 x[3];
        dc_split(f, x);
        lh = u32x4{x[2][0], x[2][1], x[0][0], x[0][1]};
        mh = u32x4{x[1][0], x[1][1], x[0][0], x[0][1]};
        hm = u32x4{x[0][0], x[0][1], x[1][0], x[1][1]};
    }
};

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

// Gates of one value head and chunk that prep's waves share
struct DcGates {
    float beta[kDcSpan];   // beta_t r_t, with k_t r_t the key (r is 1 without the norm)
    float row[kDcSpan];    // decay from the tile's start through t
    float tail[kDcSpan];   // decay behind t to the tile's end, times r_t
    float log[kDcSpan];
    float total[4];     // logs of a tile
};

template <typename IO, int D>
struct DcPrepLds {
    static constexpr int PL = DcShape<IO, D>::PL;
    static constexpr int DH = D < 256 / PL ? D : PL == 1 ? 256 : PL == 2 ? 128 : 64;  // keys at a time
    // planes of four tiles each
    unsigned char k[PL][kDcSpan * DH * 2], q[PL][kDcSpan * DH * 2];
    float ks[kDcSpan], qs[kDcSpan], kk[kDcSpan];  // r of k, of q times the scale; |r k|^2
    DcGates gates[4];
    float diag[4][16 * 20];
};

template <typename IO, int D>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaParams p, DeltaWork w)
{
    using Sh = DcShape<IO, D>;
    constexpr int KS = D / 32, NT = Sh::NT, PL = Sh::PL, C = Sh::C, CH = Sh::CH;
    constexpr int DH = DcPrepLds<IO, D>::DH, HS = DH / 32;
    static_assert(D % DH == 0, "keys in equal parts");
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

    // k and q of tile `wave`
    constexpr int VL = sizeof(IO) == 4 ? 2 : 1;  // 16-byte loads of eight entries
    u32x4 raw[2][KS][VL];
    {
        const int tok = 16 * wave + c;
        const bool in = tok < n;
        const IO *kp = static_cast<const IO *>(p.k) + b * p.k_bs + (t0 + tok) * p.k_ts + j * D + 8 * g;
        const IO *qp = static_cast<const IO *>(p.q) + b * p.q_bs + (t0 + tok) * p.q_ts + j * D + 8 * g;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int x = 0; x < VL; ++x) {
                raw[0][ks][x] = raw[1][ks][x] = u32x4{0, 0, 0, 0};
                if (in) {
                    raw[0][ks][x] = reinterpret_cast<const u32x4 *>(kp + 32 * ks)[x];
                    if (p.out)
                        raw[1][ks][x] = reinterpret_cast<const u32x4 *>(qp + 32 * ks)[x];
                }
            }
        gates_of(wave);
    }

    // K_s . K_t and K_s . Q_t of the row tile `wave`: column t of the tile, rows s. L and P share
    // their decays, which weighs more than that the last tile's wave has the most columns.
    // i: the row tile within its chunk
    const int sub = wave / NT, i0 = sub * NT, i = wave - i0;
    const int64_t at = (int64_t)b * w.chunks + span * CH;
    dc_f32x4 kk[NT], qk[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        kk[t] = qk[t] = dc_f32x4{0, 0, 0, 0};
    float sums[2] = {0.0f, 0.0f};
#pragma unroll
    for (int half = 0; half < D / DH; ++half) {
        if (half > 0)
            __syncthreads();
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int hs = 0; hs < HS; ++hs) {
                const u32x4 (&in)[VL] = raw[s][half * HS + hs];
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (sizeof(IO) == 4)
                        v[e] = __uint_as_float(in[e / 4][e % 4]);
                    else
                        v[e] = cvt_raw1<IO>(e % 2 ? in[0][e / 2] >> 16 : in[0][e / 2] & 0xffffu);
                    sums[s] += v[e] * v[e];
                }
                uint32_t part[PL][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (PL == 1) {
                        part[0][e] = in[0][e];
                    } else {
#pragma unroll
                        for (int x = 0; x < PL; ++x)
                            part[x][e] = dc_part(v[2 * e], v[2 * e + 1]);
                    }
                }
                // keys 32 hs + 8 g ..: pieces 2 g and 2 g + 1 of the eight pieces of a step
                const int tok = 16 * wave + c;
#pragma unroll
                for (int x = 0; x < PL; ++x) {
                    unsigned char *image = s ? lds.q[x] : lds.k[x];
                    *reinterpret_cast<u32x2 *>(image + dc_at<DH>(tok, 2 * hs + (g >> 1), 2 * (g & 1))) = u32x2{part[x][0], part[x][1]};
                    *reinterpret_cast<u32x2 *>(image + dc_at<DH>(tok, 2 * hs + (g >> 1), 2 * (g & 1) + 1)) = u32x2{part[x][2], part[x][3]};
                }
            }
        if (half == D / DH - 1) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const float sum = dc_sum_groups(sums[s]);
                const float r = p.use_l2 ? 1.0f / sqrtf(sum + kDeltaEps) : 1.0f;
                if (g == 0) {
                    const int tok = 16 * wave + c;
                    if (s == 0) {
                        lds.ks[tok] = r;
                        lds.kk[tok] = sum * r * r;  // NaN or inf where k's is
                    } else {
                        lds.qs[tok] = r * p.scale;
                    }
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < PL; ++x)
#pragma unroll
            for (int o16 = 0; o16 < kDcSpan * DH * 2 / 4096; ++o16) {
                const int o = (o16 * 256 + threadIdx.x) * 16;
                const int tile = o / (32 * DH), in = o - tile * (32 * DH);
                unsigned char *to = w.kq + ((at + tile / NT) * p.hq + j) * Sh::KQ + x * NT * Sh::TILE +
                                    tile % NT * Sh::TILE + half * (32 * DH) + in;
                *reinterpret_cast<u32x4 *>(to) = *reinterpret_cast<const u32x4 *>(lds.k[x] + o);
                if (p.out)
                    *reinterpret_cast<u32x4 *>(to + Sh::KQ / 2) = *reinterpret_cast<const u32x4 *>(lds.q[x] + o);
            }
        auto operand = [&](const unsigned char (&image)[PL][kDcSpan * DH * 2], int tile, int hs, u32x4 (&op)[PL]) {
#pragma unroll
            for (int x = 0; x < PL; ++x)
                op[x] = dc_ld_op<DH>(image[x], tile, hs, lane);
        };
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (t <= i)
#pragma unroll
                for (int hs = 0; hs < HS; ++hs) {
                    u32x4 a[PL], o[PL];
                    operand(lds.k, i0 + t, hs, a);
                    operand(lds.k, i0 + i, hs, o);
                    dc_each<PL, PL>([&](int x, int y) { kk[t] = dc_mfma(a[x], o[y], kk[t]); });
                    if (p.out) {
                        operand(lds.q, i0 + i, hs, o);
                        dc_each<PL, PL>([&](int x, int y) { qk[t] = dc_mfma(a[x], o[y], qk[t]); });
                    }
                }
    }

    for (int h0 = 0; h0 < G; h0 += 4) {
        if (h0 + wave < G) {  // gates of four heads at once, lane = token
            const int h = j * G + h0 + wave;
            const bool in = lane < n;
            if (h0 > 0)
                gates_of(h0 + wave);
            const float ks = lds.ks[lane], qs = lds.qs[lane], kk2 = lds.kk[lane];
            const float bk = beta * kk2;
            // (a q reaches no output but its own)
            const bool bad = in && !(lg <= 0.0f && kk2 < __builtin_inff() && bk >= -1.0001f && bk <= 2.0001f);
            const int mine = lane / C;  // chunk
            const uint64_t of_mine = (C == 64 ? ~(uint64_t)0 : (((uint64_t)1 << (C % 64)) - 1)) << (mine * C % 64);
            const float kind = __ballot(bad) & of_mine ? 1.0f : 0.0f;
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
#pragma unroll
            for (int jt = 0; jt < NT - 1; ++jt) {
                if (jt >= i)
                    break;
                float mid = 0.0f;
                for (int m = jt + 1; m < i; ++m)
                    mid += s.total[i0 + m];
                const float f = row * expf(mid);
                const dc_f32x4 tail = *reinterpret_cast<const dc_f32x4 *>(&s.tail[16 * (i0 + jt) + 4 * g]) * f;
                dc_st_tile(to + Sh::l_tile(i, jt), lane, tail * kk[jt] * -own);
                if (p.out)
                    dc_st_tile(to + Sh::p_tile(i, jt), lane, tail * qk[jt]);
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
                x[r] = 4 * g + r < c ? d * x[r] * own : 0.0f;
                y[r] = 4 * g + r <= c ? d * y[r] : 0.0f;
            }
            if (p.out)
                dc_st_tile(to + Sh::p_tile(i, i), lane, y);
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
            dc_st_tile(to + i * kDcTile, lane, x);
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

// Values of four tokens 4 g + r of tile i, column c of the wave's 16, from its token rows in LDS
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
};

// A workgroup: W waves of 16 value columns each, of value head h, batch entry b. Up to four have a wave beside them
// that fetches (a chunk's loads, issued by waves alone on their SIMDs, cost them 22 us of 300, and in front of a
// chunk they would wait for their own outputs too); eight hide the issue behind each other, and a ninth would
// leave 168 registers a wave (1024 tokens, 16 heads of 256, 8 rows: 303 us for 220).
constexpr bool dc_loader(int waves) { return waves <= 4; }

template <typename IO, int D, int W, bool OUT>
__global__ __launch_bounds__(64 * (W + dc_loader(W)), W > 4 ? 2 : 1) void delta_sweep_kernel(DeltaParams p, DeltaWork w, int swizzle)
{
    using Sh = DcShape<IO, D>;
    constexpr int KS = D / 32, KT = D / 16, NT = Sh::NT, PL = Sh::PL, C = Sh::C, NP = NT / 2;
    constexpr int TILES = D / (16 * W);                // workgroups a head
    constexpr int KQ = Sh::KQ, VP = 16 * sizeof(IO);   // bytes of K and Q, of a token's values of a wave
    constexpr int BUF = Sh::buffer(W), NB = Sh::buffers(W);  // bytes of a chunk in LDS, chunks
    constexpr int PLANE = NT * Sh::TILE;
    static_assert(TILES * 16 * W == D && NB * BUF <= 160 * 1024, "value columns of a head; LDS");
    __shared__ __attribute__((aligned(16))) unsigned char lds[NB * BUF];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    // workgroups are dealt out over eight XCDs: those of one q head go to the same one
    const uint32_t id = swizzle ? (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3) : blockIdx.x;
    const int64_t bh = id / TILES;
    const int b = (int)(bh / p.hv), h = (int)(bh - (int64_t)b * p.hv);
    const int v0 = (int)(id - bh * TILES) * (16 * W) + wave * 16;
    const int j = h / (p.hv / p.hq);
    const int pool = p.idx ? p.idx[b] : b;
    const int len = pool < 0 ? 0 : (p.ctx ? clamp_len(p.ctx[b], p.seq_len) : p.seq_len);
    const int mine = min(len - w.chunk0 * C, w.chunks * C);  // tokens of the segment
    if (len <= 0 || (mine <= 0 && !(w.last && p.update && !w.first)))
        return;
    const int chunks = mine > 0 ? (mine + C - 1) / C : 0;

    // What prep left of a chunk, and its values, go to LDS past the registers, 1 KiB an instruction,
    // while the chunk before it is worked on
    constexpr bool LOADER = dc_loader(W);
    constexpr int FW = LOADER ? 1 : W;  // waves that fetch
    const int mine_of = LOADER ? 0 : wave;
    const unsigned char *kq = w.kq + ((int64_t)b * w.chunks * p.hq + j) * KQ + lane * 16;
    const unsigned char *hd = w.head + ((int64_t)b * w.chunks * p.hv + h) * Sh::HEAD + lane * 16;
    const int64_t kq_step = (int64_t)p.hq * KQ, hd_step = (int64_t)p.hv * Sh::HEAD;
    constexpr int VL = VP / 16, VR = 64 / VL;  // lanes a token's values, tokens an instruction
    constexpr int QK = OUT ? KQ : KQ / 2, HD = OUT ? Sh::HEAD : (Sh::P + 1023) / 1024 * 1024;
    static_assert(C % VR == 0 && QK % 1024 == 0, "whole instructions");
    const IO *vp = static_cast<const IO *>(p.v) + b * p.v_bs + (int64_t)w.chunk0 * C * p.v_ts +
                   (int64_t)h * D + (LOADER ? v0 - wave * 16 : v0) + 16 / sizeof(IO) * (lane % VL);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char *)lds;
    // part 0 .. 3 of four (the CU takes 64 bytes a cycle: issued at once, they would stall the wave)
    auto fetch = [&](int ch, int part) {
        const uint32_t to = lds0 + ch % NB * BUF;
#pragma unroll
        for (int q = 0; q < C / VR; ++q)
            if (q % 4 == part) {
                const int t = ch * C + q * VR + lane / VL;  // rows behind the end repeat the last
                const IO *from = vp + (int64_t)min(t, mine - 1) * p.v_ts;
#pragma unroll
                for (int x = 0; x < (LOADER ? W : 1); ++x)
                    dc_to_lds(reinterpret_cast<const unsigned char *>(from + 16 * x),
                              to + KQ + Sh::HEAD + (mine_of + x) * (C * VP) + q * 1024);
            }
        const unsigned char *from = kq + ch * kq_step + mine_of * 1024;
#pragma unroll
        for (int o = 0; o < QK; o += FW * 1024)
            if (o / (FW * 1024) % 4 == part && (o + FW * 1024 <= QK || o + mine_of * 1024 < QK))
                dc_to_lds(from + o, to + mine_of * 1024 + o);
        from = hd + ch * hd_step + mine_of * 1024;
#pragma unroll
        for (int o = 0; o < HD; o += FW * 1024)
            if (o / (FW * 1024) % 4 == part && (o + FW * 1024 <= HD || o + mine_of * 1024 < HD))
                dc_to_lds(from + o, to + KQ + mine_of * 1024 + o);
    };
    auto fetch_all = [&](int ch) {
#pragma unroll
        for (int part = 0; part < 4; ++part)
            fetch(ch, part);
    };
    // In front of a chunk its LDS is filled (by every wave: behind the barrier), the other one read
    auto arrive = [&](int ch) {
        if (NB == 1) {
            __syncthreads();
            fetch_all(ch);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    };
    if (NB == 2 && chunks > 0 && (!LOADER || wave == W))
        fetch_all(0);
    if (LOADER && wave == W) {
        for (int ch = 0; ch < chunks; ++ch) {
            arrive(ch);
            if (NB == 2 && ch + 1 < chunks)
                fetch_all(ch + 1);
        }
        return;
    }

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

    for (int ch = 0; ch < chunks; ++ch) {
        if (!LOADER) {
            arrive(ch);
        } else {
            if (NB == 1)
                __syncthreads();
            __syncthreads();
        }
        unsigned char *image = lds + ch % NB * BUF;
        const unsigned char *blk = image + KQ;
        unsigned char *rows = image + KQ + Sh::HEAD + wave * (C * VP);  // values of the wave's columns
        const float *scal = reinterpret_cast<const float *>(blk + Sh::SCALARS);
        const int t0 = ch * C, n_tok = min(mine - t0, C);
        const int64_t tok0 = (int64_t)w.chunk0 * C + t0;
        const bool ahead = !LOADER && NB == 2 && ch + 1 < chunks;
        if (ahead)
            fetch(ch + 1, 0);
        DcValues<IO, VP> v[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i)
            v[i].load(rows, i, lane);
        if (n_tok < C) {  // what was read in the place of tokens behind the end
#pragma unroll
            for (int i = 0; i < NT; ++i)
                v[i].keep(n_tok - (16 * i + 4 * g));
        }
        const float all = scal[kScMisc * C];
        bool slow = __builtin_amdgcn_readfirstlane(__float_as_uint(scal[kScMisc * C + 1])) != 0;  // the same in every lane
        dc_f32x4 X[NT], O[NT], Q[NT];
        if (!slow) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
                X[i] = O[i] = dc_f32x4{0, 0, 0, 0};
            auto operand = [&](const unsigned char *at, int i, int ks, u32x4 (&op)[PL]) {
#pragma unroll
                for (int x = 0; x < PL; ++x)
                    op[x] = dc_ld_op<D>(at + x * PLANE, i, ks, lane);
            };
            u32x4 kf[NT][PL];
#pragma unroll
            for (int i = 0; i < NT; ++i)
                operand(image, i, 0, kf[i]);
            // S0 k and S0 q
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                u32x4 sp[3], qf[NT][PL], kn[NT][PL];
                dc_split2(S[2 * ks], S[2 * ks + 1], sp);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if (OUT)
                        operand(image + KQ / 2, i, ks, qf[i]);
                    if (ks + 1 < KS)
                        operand(image, i, ks + 1, kn[i]);
                }
                dc_each<PL, 3>([&](int x, int y) {
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        X[i] = dc_mfma(kf[i][x], sp[y], X[i]);
                });
                if (OUT)
                    dc_each<3, PL>([&](int x, int y) {
#pragma unroll
                        for (int i = 0; i < NT; ++i)
                            O[i] = dc_mfma(sp[x], qf[i][y], O[i]);
                    });
                if (ks + 1 < KS)
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int x = 0; x < PL; ++x)
                            kf[i][x] = kn[i][x];
            }
            if (ahead)
                fetch(ch + 1, 1);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const dc_f32x4 beta = *reinterpret_cast<const dc_f32x4 *>(scal + kScBeta * C + 16 * i + 4 * g);
                const dc_f32x4 gk = *reinterpret_cast<const dc_f32x4 *>(scal + kScGk * C + 16 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    X[i][r] = beta[r] * (v[i][r] - gk[r] * X[i][r]);
            }
            if (ahead)
                fetch(ch + 1, 2);
            // U, tile after tile, and what each leaves of the others' X and adds to the outputs
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                DcTile m;
                m.load(blk + i * kDcTile, lane);
                const DcOther x(X[i]);
                dc_f32x4 u = {0, 0, 0, 0};
                u = dc_mfma(m.hl, x.lh, u);
                u = dc_mfma(m.hm, x.mh, u);
                u = dc_mfma(m.hm, x.hm, u);
                X[i] = u;
                const DcOther uo(u);
                DcTile l[NT];
#pragma unroll
                for (int t = i + 1; t < NT; ++t)
                    l[t].load(blk + Sh::l_tile(t, i), lane);
#pragma unroll
                for (int t = i + 1; t < NT; ++t)
                    X[t] = dc_mfma(l[t].hl, uo.lh, X[t]);
#pragma unroll
                for (int t = i + 1; t < NT; ++t)
                    X[t] = dc_mfma(l[t].hm, uo.mh, X[t]);
#pragma unroll
                for (int t = i + 1; t < NT; ++t)
                    X[t] = dc_mfma(l[t].hm, uo.hm, X[t]);
                if (OUT) {
#pragma unroll
                    for (int t = i; t < NT; ++t) {
                        DcTile pt;
                        pt.load(blk + Sh::p_tile(t, i), lane);
                        if (i == 0)
                            Q[t] = dc_f32x4{0, 0, 0, 0};
                        Q[t] = dc_mfma(uo.lh, pt.hl, Q[t]);
                        Q[t] = dc_mfma(uo.mh, pt.hm, Q[t]);
                        Q[t] = dc_mfma(uo.hm, pt.hm, Q[t]);
                    }
                }
            }
            // what is not finite in a column's state, values or U before has reached all of the last tile
            bool bad = false;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                bad |= !(fabsf(X[NT - 1][r]) < __builtin_inff());
            slow = __ballot(bad) != 0;
        }

        if (!slow) {
            if (ahead)
                fetch(ch + 1, 3);
            if (OUT) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const float go = scal[kScGo * C + 16 * i + c], qo = scal[kScQo * C + 16 * i + c];
                    float o[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        o[r] = go * O[i][r] + qo * Q[i][r];
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
                const dc_f32x4 w0 = *reinterpret_cast<const dc_f32x4 *>(scal + kScWk * C + 32 * s + 4 * g);
                const dc_f32x4 w1 = *reinterpret_cast<const dc_f32x4 *>(scal + kScWk * C + 32 * s + 16 + 4 * g);
                u32x4 wu[3];
                dc_split2(X[2 * s] * w0, X[2 * s + 1] * w1, wu);
                constexpr int AT = PL > 1 || KT < 4 ? 2 : 4;  // tiles at a time
#pragma unroll
                for (int n0 = 0; n0 < KT; n0 += AT) {
                    u32x4 kt[AT][PL];
#pragma unroll
                    for (int n = 0; n < AT; ++n)
#pragma unroll
                        for (int x = 0; x < PL; ++x)
                            kt[n][x] = dc_ld_kt<D>(image + x * PLANE, n0 + n, s, lane);
                    dc_each<PL, 3>([&](int x, int y) {
#pragma unroll
                        for (int n = 0; n < AT; ++n)
                            S[n0 + n] = dc_mfma(kt[n][x], wu[y], S[n0 + n]);
                    });
                }
            }
        } else {
            if (ahead) {  // some of it again where U was formed
#pragma unroll
                for (int part = 1; part < 4; ++part)
                    fetch(ch + 1, part);
            }
            // token by token
            auto ld_keys = [&](const unsigned char *at, int t, int n) {
                dc_f32x4 k;
#pragma unroll
                for (int x = PL - 1; x >= 0; --x) {
                    const u32x2 bits = *reinterpret_cast<const u32x2 *>(at + x * PLANE + dc_at<D>(t, n, g));
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float f = __uint_as_float(r % 2 ? bits[r / 2] & 0xffff0000u : bits[r / 2] << 16);
                        k[r] = x < PL - 1 ? k[r] + f : f;
                    }
                }
                return k;
            };
            for (int t = 0; t < n_tok; ++t) {
                const float alpha = scal[kScAlpha * C + t], ks = scal[kScKs * C + t];
                const float beta = scal[kScBeta * C + t], qs = scal[kScQo * C + t];
                const float vt = ld_elem<IO>(rows + t * VP, c);
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
                const float u = beta * (vt - alpha * (sum * ks));
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
                    o = dc_sum_groups(o) * qs;
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
#pragma unroll
    for (int n = 0; n < KT; ++n) {
        const int o = (v0 + c) * D + 16 * n + 4 * g;
        const float s[4] = {S[n][0], S[n][1], S[n][2], S[n][3]};
        if (!w.last) {
            *reinterpret_cast<dc_f32x4 *>(carry + o) = S[n];
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
    if (!launchable(groups, 64 * (W + dc_loader(W))))
        return hipErrorInvalidConfiguration;
    const uint32_t n = (uint32_t)groups;
    if (p.out)
        delta_sweep_kernel<IO, D, W, true><<<dim3(n), 64 * (W + dc_loader(W)), 0, stream>>>(p, w, n % 8 == 0);
    else
        delta_sweep_kernel<IO, D, W, false><<<dim3(n), 64 * (W + dc_loader(W)), 0, stream>>>(p, w, n % 8 == 0);
    return hipGetLastError();
}

template <typename IO, int D>
hipError_t launch_delta_chunks_d(const DeltaParams &p, const DeltaPlan &plan, hipStream_t stream)
{
    using Sh = DcShape<IO, D>;
    constexpr int W = D == 32 ? 2 : 4, WIDE = D >= 128 && Sh::buffers(8) == Sh::buffers(W) ? 8 : W;
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
