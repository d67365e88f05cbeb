// Log probabilities of given tokens, the entropy of their distributions and the
// most probable alternatives, from logits, in one pass over them:
//   lse = m + log s,  s = sum e^(x - m);  entropy = log s - (sum e^(x - m) (x - m)) / s
// Each lane keeps m, s and the weighted sum t of what it has seen and rescales
// them when m grows (t <- e^d (t + d s), d = m_old - m_new). HBM bounds it.
//
// The k largest logits of a wave stand in its lanes, entry i in lane i, ordered
// by (value descending, index ascending). A tile of 64 x 16 logits is compared
// with the last of them by the lanes' maxima: most tiles after the first few hold
// nothing that gets in. The k-th largest of the 64 lanes' maxima over all tiles so far
// bounds the k-th largest logit from below, which leaves little more than k to insert.
//
// A row goes to one workgroup where there are rows enough, else to several:
// their sums and lists go through the workspace to a second launch, one
// workgroup a row, which orders them in a fixed order. So results do not
// depend on which workgroup comes first.
#include <limits.h>
#include <math.h>

#include "ssu_device.h"
#include "ssu_dpp.h"
#include "ssu_internal.h"

namespace ssu {
namespace {

constexpr int kTile = 16;          // logits a lane takes at once
constexpr int kWaves = 4;          // waves of a workgroup
constexpr int kMaxTop = SSU_MAX_TOP;
constexpr float kFloor = -200.0f;  // e^x is 0 in fp32 far above

// What a part of a row comes to; s is NaN where a logit is NaN or +inf.
struct Sums {
    float m, s, t;
};

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// An m that may be subtracted: one of -inf has no logit to it
__device__ __forceinline__ float anchor(float m) { return m == neg_inf() ? 0.0f : m; }

// e^x by the hardware's 2^x (within an ulp; the argument's own rounding is |x| 2^-24 of the value)
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

__device__ __forceinline__ void rescale(Sums &a, float m)
{
    const float d = fmaxf(a.m - anchor(m), kFloor), e = exp_of(d);
    a.t = e * (a.t + d * a.s);
    a.s *= e;
    a.m = m;
}

__device__ __forceinline__ Sums join(Sums a, Sums b)
{
    const float m = fmaxf(a.m, b.m);
    rescale(a, m);
    rescale(b, m);
    return {m, a.s + b.s, a.t + b.t};
}

__device__ __forceinline__ bool better(float x, int i, float y, int j)
{
    return x > y || (x == y && i < j);
}

// The k largest of a wave: lane i < k holds entry i.
struct Top {
    float v;
    int id;
    float last_v;  // entry k - 1, the same in every lane
    int last_id;

    __device__ __forceinline__ void clear()
    {
        v = last_v = neg_inf();
        id = last_id = INT_MAX;
    }
    // x, i the same in every lane
    __device__ __forceinline__ void insert(float x, int i, int k, int lane)
    {
        const int at = __popcll(__ballot(lane < k && better(v, id, x, i)));
        // DPP wave_shr:1, a lane's value from the lane before it
        const float pv = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x138, 0xF, 0xF, false));
        const int pi = __builtin_amdgcn_update_dpp(0, id, 0x138, 0xF, 0xF, false);
        v = lane == at ? x : lane > at ? pv : v;
        id = lane == at ? i : lane > at ? pi : id;
        last_v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), k - 1));
        last_id = __builtin_amdgcn_readlane(id, k - 1);
    }
};

// k-th largest of the lanes' values (k <= 64), -inf if it is not finite: bit after bit of
// the largest bound that k lanes reach, over bits that order as the values do.
__device__ __forceinline__ float kth_of_lanes(float x, int k)
{
    const uint32_t b = __float_as_uint(x);
    const uint32_t key = b & 0x80000000u ? ~b : b | 0x80000000u;
    uint32_t bound = 0;
    for (int bit = 31; bit >= 16; --bit) {  // the low bits are left at 0: still a bound from below
        const uint32_t next = bound | (1u << bit);
        if (__popcll(__ballot(key >= next)) >= k)
            bound = next;
    }
    const float f = __uint_as_float(bound & 0x80000000u ? bound ^ 0x80000000u : ~bound);
    return f <= 3.0e38f && f >= -3.0e38f ? f : neg_inf();
}

template <typename T>
struct LogitTile {
    static constexpr int VE = sizeof(T) == 4 ? 4 : 8;  // logits of a 16-byte load
    static constexpr int NL = kTile / VE;
    u32x4 w[NL];

    // the index of element e of load l, from the tile's first
    __device__ static __forceinline__ int at(int lane, int l, int e) { return (l * 64 + lane) * VE + e; }

    template <bool VEC>
    __device__ __forceinline__ void load(const T *p, int left, int lane)
    {
#pragma unroll
        for (int l = 0; l < NL; ++l) {
            const int i = at(lane, l, 0);
            if (VEC && i + VE <= left) {
                w[l] = *reinterpret_cast<const u32x4 *>(p + i);
            } else {
                u32x4 r = {};
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    if (i + e < left) {
                        if constexpr (sizeof(T) == 4)
                            r[e] = reinterpret_cast<const uint32_t *>(p)[i + e];
                        else
                            r[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[i + e] << (16 * (e % 2));
                    }
                }
                w[l] = r;
            }
        }
    }
    __device__ __forceinline__ float value(int l, int e) const
    {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[l][e]);
        else
            return cvt_raw1<T>(e % 2 ? w[l][e / 2] >> 16 : w[l][e / 2] & 0xffffu);
    }
};

// Logits [begin, end) of a row by one wave, every `step` th tile from `begin`.
template <typename T, bool VEC>
__device__ void wave_pass(const T *row, int begin, int end, int step, int k, int lane, Sums &sums,
                          Top &top)
{
    using Tile = LogitTile<T>;
    sums = {neg_inf(), 0.0f, 0.0f};
    top.clear();
    constexpr int N = 64 * kTile;
    Tile next;
    if (begin < end)
        next.template load<VEC>(row + begin, end - begin, lane);
    float most = neg_inf();   // of the lane, over all tiles
    float bound = neg_inf();  // at least k logits reach it
    for (int64_t base = begin; base < end; base += (int64_t)step * N) {
        const Tile cur = next;
        const int left = end - (int)base;
        if (base + (int64_t)step * N < end)
            next.template load<VEC>(row + base + (int64_t)step * N, left - step * N, lane);
        float x[kTile];
#pragma unroll
        for (int l = 0; l < Tile::NL; ++l)
#pragma unroll
            for (int e = 0; e < Tile::VE; ++e)
                x[l * Tile::VE + e] = cur.value(l, e);
        if (left < N) {
#pragma unroll
            for (int l = 0; l < Tile::NL; ++l)
#pragma unroll
                for (int e = 0; e < Tile::VE; ++e)
                    if (Tile::at(lane, l, e) >= left)
                        x[l * Tile::VE + e] = neg_inf();
        }
        float m = neg_inf();
#pragma unroll
        for (int e = 0; e < kTile; ++e)
            m = fmaxf(m, x[e]);
        if (m > sums.m)
            rescale(sums, m);
        const float from = anchor(sums.m);
#pragma unroll
        for (int e = 0; e < kTile; ++e) {
            const float d = x[e] - from, p = exp_of(d);  // a NaN stays one in s
            sums.s += p;
            sums.t += p * fmaxf(d, kFloor);
        }
        if (k > 0 && __ballot(m >= bound && m >= top.last_v)) {
            most = fmaxf(most, m);
            bound = fmaxf(bound, kth_of_lanes(most, k));
#pragma unroll
            for (int l = 0; l < Tile::NL; ++l)
#pragma unroll
                for (int e = 0; e < Tile::VE; ++e) {
                    const float v = x[l * Tile::VE + e];
                    const int at = Tile::at(lane, l, e), id = (int)base + at;
                    const bool in = at < left && v >= bound;
                    uint64_t todo = __ballot(in && better(v, id, top.last_v, top.last_id));
                    while (todo) {
                        const int one = __ffsll((unsigned long long)todo) - 1;
                        top.insert(__builtin_bit_cast(float, __builtin_amdgcn_readlane(
                                                                 __builtin_bit_cast(int, v), one)),
                                   __builtin_amdgcn_readlane(id, one), k, lane);
                        todo &= todo - 1;
                        todo &= __ballot(in && better(v, id, top.last_v, top.last_id));
                    }
                }
        }
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        Sums b;
        b.m = __shfl_xor(sums.m, o, 64);
        b.s = __shfl_xor(sums.s, o, 64);
        b.t = __shfl_xor(sums.t, o, 64);
        sums = join(sums, b);
    }
}

__device__ __forceinline__ bool row_live(const LogprobParams &p, int64_t row)
{
    const int b = (int)(row / p.num_tokens), t = (int)(row - (int64_t)b * p.num_tokens);
    return (!p.idx || p.idx[b] >= 0) && (!p.ctx || t < p.ctx[b]);
}

// The answers of a row from its sums; lane i < k holds entry i of the list.
template <typename T>
__device__ void write_row(const LogprobParams &p, int64_t row, const T *logits, const Sums &a,
                          float v, int id, int lane)
{
    const float nan = __builtin_nanf("");
    const float log_s = logf(a.s);
    const bool bad = a.s != a.s;
    // x - lse as (x - m) - log s: exact differences of large logits first
    auto logprob = [&](float x) {
        return bad ? nan : x == neg_inf() ? neg_inf() : (x - a.m) - log_s;
    };
    if (lane == 0) {
        const int tok = p.tokens[row];
        p.logprobs[row] = tok < 0 || tok >= p.vocab ? neg_inf() : logprob(ld_elem<T>(logits, tok));
        if (p.entropy)
            p.entropy[row] = bad ? nan : a.m == neg_inf() ? 0.0f : fmaxf(log_s - a.t / a.s, 0.0f);
    }
    if (lane < p.top) {
        const bool none = id == INT_MAX;  // only beside NaN
        p.top_ids[row * p.top + lane] = none ? -1 : id;
        p.top_logprobs[row * p.top + lane] = none ? nan : logprob(v);
    }
}

__device__ void write_padding(const LogprobParams &p, int64_t row, int lane)
{
    if (lane == 0) {
        p.logprobs[row] = 0.0f;
        if (p.entropy)
            p.entropy[row] = 0.0f;
    }
    if (lane < p.top) {
        p.top_ids[row * p.top + lane] = -1;
        p.top_logprobs[row * p.top + lane] = 0.0f;
    }
}

// The k best of `parts` ordered lists of k in (vs, ids), each entry's place being
// the number of better ones; the first wave writes them to its lanes.
__device__ void place_lists(const float *vs, const int *ids, int parts, int k, float *out_v,
                            int *out_id)
{
    const int n = parts * k;
    for (int i = threadIdx.x; i < k; i += blockDim.x) {
        out_v[i] = neg_inf();
        out_id[i] = INT_MAX;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const float x = vs[i];
        const int id = ids[i];
        int at = i % k;  // those before it in its own list
        for (int q = 0; q < parts && at < k; ++q) {
            if (q == i / k)
                continue;
            for (int j = 0; j < k && better(vs[q * k + j], ids[q * k + j], x, id); ++j)
                ++at;
        }
        if (at < k && id != INT_MAX) {
            out_v[at] = x;
            out_id[at] = id;
        }
    }
    __syncthreads();
}

// Part of a row in the workspace: its sums, then k values, then k ids.
__host__ __device__ inline int64_t part_words(int64_t top) { return 4 + 2 * top; }  // one word is left out

template <typename T, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void logprobs_kernel(LogprobParams p, int parts, int part)
{
    __shared__ Sums sums_of[kWaves];
    __shared__ float vs[kWaves * kMaxTop], best_v[kMaxTop];
    __shared__ int ids[kWaves * kMaxTop], best_id[kMaxTop];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x / (uint32_t)parts;
    const int which = (int)(blockIdx.x - (uint32_t)(row * parts));
    if (!row_live(p, row)) {
        if (which == 0 && wave == 0)
            write_padding(p, row, lane);
        return;
    }
    const int b = (int)(row / p.num_tokens), t = (int)(row - (int64_t)b * p.num_tokens);
    const T *logits = static_cast<const T *>(p.logits) + b * p.l_bs + t * p.l_rs;
    const int64_t begin = (int64_t)which * part;
    const int end = (int)min((int64_t)p.vocab, begin + part);
    Sums sums;
    Top top;
    const int64_t mine = begin + (int64_t)wave * 64 * kTile;
    wave_pass<T, VEC>(logits, (int)min(mine, (int64_t)end), end, kWaves, p.top, lane, sums, top);
    if (lane == 0)
        sums_of[wave] = sums;
    if (lane < p.top) {
        vs[wave * p.top + lane] = top.v;
        ids[wave * p.top + lane] = top.id;
    }
    __syncthreads();
    if (p.top > 0)
        place_lists(vs, ids, kWaves, p.top, best_v, best_id);
    if (wave != 0)
        return;
    Sums a = sums_of[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
        a = join(a, sums_of[w]);
    const float v = lane < p.top ? best_v[lane] : 0.0f;
    const int id = lane < p.top ? best_id[lane] : 0;
    if (parts == 1) {
        write_row<T>(p, row, logits, a, v, id, lane);
        return;
    }
    float *w = static_cast<float *>(p.workspace) + (row * parts + which) * part_words(p.top);
    if (lane == 0)
        *reinterpret_cast<Sums *>(w) = a;
    if (lane < p.top) {
        w[4 + lane] = v;
        reinterpret_cast<int *>(w)[4 + p.top + lane] = id;
    }
}

constexpr int kMaxParts = 64;

template <typename T>
__global__ __launch_bounds__(256) void logprobs_join_kernel(LogprobParams p, int parts)
{
    __shared__ float vs[kMaxParts * kMaxTop], best_v[kMaxTop];
    __shared__ int ids[kMaxParts * kMaxTop], best_id[kMaxTop];
    const int lane = threadIdx.x & 63;
    const int64_t row = blockIdx.x;
    if (!row_live(p, row))
        return;
    const float *w = static_cast<const float *>(p.workspace) + row * parts * part_words(p.top);
    const int64_t pw = part_words(p.top);
    for (int i = threadIdx.x; i < parts * p.top; i += blockDim.x) {
        const int q = i / p.top, j = i - q * p.top;
        vs[i] = w[q * pw + 4 + j];
        ids[i] = reinterpret_cast<const int *>(w)[q * pw + 4 + p.top + j];
    }
    __syncthreads();
    if (p.top > 0)
        place_lists(vs, ids, parts, p.top, best_v, best_id);
    if (threadIdx.x >= 64)
        return;
    Sums a = {neg_inf(), 0.0f, 0.0f};
    if (lane < parts)
        a = *reinterpret_cast<const Sums *>(w + lane * pw);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        Sums b;
        b.m = __shfl_xor(a.m, o, 64);
        b.s = __shfl_xor(a.s, o, 64);
        b.t = __shfl_xor(a.t, o, 64);
        a = join(a, b);
    }
    const int b = (int)(row / p.num_tokens), t = (int)(row - (int64_t)b * p.num_tokens);
    const T *logits = static_cast<const T *>(p.logits) + b * p.l_bs + t * p.l_rs;
    write_row<T>(p, row, logits, a, lane < p.top ? best_v[lane] : 0.0f,
                 lane < p.top ? best_id[lane] : 0, lane);
}

// Workgroups a row takes: enough to fill the GPU, each with a tile a wave at least.
int logprobs_parts(int64_t rows, int64_t vocab)
{
    const int64_t most = (vocab + kWaves * 64 * kTile - 1) / (kWaves * 64 * kTile);
    int64_t parts = rows > 0 ? 1024 / rows : 1;
    parts = parts < 1 ? 1 : parts > kMaxParts ? kMaxParts : parts;
    return (int)(parts < most ? parts : most);
}

template <typename T>
hipError_t launch_logprobs_t(const LogprobParams &p, hipStream_t stream)
{
    const int64_t rows = (int64_t)p.batch * p.num_tokens;
    const int parts = logprobs_parts(rows, p.vocab);
    const int round = kWaves * 64 * kTile;
    const int part = (int)((((int64_t)p.vocab + parts - 1) / parts + round - 1) / round * round);
    if (!launchable((__int128)rows * parts, 64 * kWaves))
        return hipErrorInvalidConfiguration;
    const int64_t e = sizeof(T);
    const bool vec = ((uintptr_t)p.logits | (uintptr_t)(p.l_bs * e) | (uintptr_t)(p.l_rs * e)) % 16 == 0;
    const dim3 grid((uint32_t)(rows * parts));
    if (vec)
        logprobs_kernel<T, true><<<grid, 64 * kWaves, 0, stream>>>(p, parts, part);
    else
        logprobs_kernel<T, false><<<grid, 64 * kWaves, 0, stream>>>(p, parts, part);
    if (parts > 1)
        logprobs_join_kernel<T><<<dim3((uint32_t)rows), 256, 0, stream>>>(p, parts);
    return hipGetLastError();
}

}  // namespace

int64_t logprobs_workspace_bytes(int64_t rows, int64_t vocab, int64_t top)
{
    const int parts = logprobs_parts(rows, vocab);
    return parts > 1 ? 4 * rows * parts * part_words(top) : 0;
}

hipError_t launch_logprobs(const LogprobParams &p, hipStream_t stream)
{
    (void)hipGetLastError();  // report only this launch's status
    switch (p.dtype) {
    case kF32: return launch_logprobs_t<float>(p, stream);
    case kF16: return launch_logprobs_t<_Float16>(p, stream);
    default: return launch_logprobs_t<bf16_t>(p, stream);
    }
}

}  // namespace ssu
