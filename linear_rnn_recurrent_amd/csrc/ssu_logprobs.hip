// Log probabilities of given tokens, the entropy of their distributions and the
// most probable alternatives, from logits, in one pass over them:
//   lse = m + log s,  s = sum e^(x - m);  entropy = log s - (sum e^(x - m) (x - m)) / s
// Each lane keeps m, s and the weighted sum t of what it has seen and rescales
// them when m grows (t <- e^d (t + d s), d = m_old - m_new).
// The vector ALU bounds 16 bits, some 15 instructions a logit, eight the least: 2039 rows of
// 32000 bf16 take 38.8 us (131 MB, 3.4 TB/s) with 3 alternatives, 56 with 20. 128 of 131072 fp32
// take 19.3 us with one (3.5 TB/s), 28.1 with 20; a row alone 11, two launches and the
// chain of its wave's tiles.
//
// The k largest logits of a wave stand in its lanes, entry i in lane i, as keys that
// order by (value descending, index ascending). A tile of 64 x 16 logits is compared
// with the last of them by the lanes' maxima: most tiles after the first few hold
// nothing that gets in. The k-th largest of the 64 lanes' maxima over all tiles so far
// bounds the k-th largest logit from below, which leaves little more than k to insert;
// the best bound of a workgroup's waves holds for all of them.
//
// A row goes to one workgroup where there are rows enough, else to several:
// their sums and lists go through the workspace to a second launch, one
// workgroup a row, which orders them in a fixed order. So results do not
// depend on which workgroup comes first.
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

// Of a wave: the lanes' maximum first, so that each lane rescales once
__device__ __forceinline__ float wave_max(float v)
{
    v = fmaxf(v, dpp_f32<0xB1>(v));   // quad_perm [1,0,3,2]
    v = fmaxf(v, dpp_f32<0x4E>(v));   // quad_perm [2,3,0,1]
    v = fmaxf(v, dpp_f32<0x141>(v));  // row_half_mirror
    v = fmaxf(v, dpp_f32<0x140>(v));  // row_mirror
    const int u = __builtin_bit_cast(int, v);
    return fmaxf(fmaxf(__builtin_bit_cast(float, __builtin_amdgcn_readlane(u, 0)),
                       __builtin_bit_cast(float, __builtin_amdgcn_readlane(u, 16))),
                 fmaxf(__builtin_bit_cast(float, __builtin_amdgcn_readlane(u, 32)),
                       __builtin_bit_cast(float, __builtin_amdgcn_readlane(u, 48))));
}
__device__ __forceinline__ Sums wave_join(Sums a)
{
    rescale(a, wave_max(a.m));
    return {a.m, wave_sum(a.s), wave_sum(a.t)};
}

// Bits that order as the values do (-0 as 0)
__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_order(uint32_t o)
{
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ float next_above(float x) { return of_order(order_of(x) + 1); }

// A logit and its index as one number, the larger the better; 0: none.
typedef uint64_t Key;
__device__ __forceinline__ Key key_of(float x, int i) { return (Key)order_of(x) << 32 | ~(uint32_t)i; }
__device__ __forceinline__ float logit_of(Key k) { return of_order((uint32_t)(k >> 32)); }
__device__ __forceinline__ int index_of(Key k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ Key lane_key(Key k, int lane)  // of lane `lane`, the same in every lane
{
    return (Key)(uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, lane);
}

// The k largest of a wave: lane i < k holds entry i. Candidates are gathered in LDS and
// ranked against the list and each other, 64 - k at a time, when there are some or at the
// end: no chain from one to the next.
constexpr int kGather = 128;  // candidates that wait for the next tile's at most
struct TopLds {
    Key got[64 * kTile + kGather];
    Key list[kMaxTop];
};

__device__ __forceinline__ void wave_lds_fence()  // LDS writes of the wave's lanes before its reads
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

struct Top {
    Key key;
    Key last;  // entry k - 1, the same in every lane

    // the first n candidates of lds, of which those below `bound` (k logits reach it) are out
    __device__ void take(TopLds &lds, int n, float bound, int k, int lane)
    {
        const Key least = (Key)order_of(bound) << 32;
        int left = 0;
        for (int i = 0; i < n; i += 64) {
            wave_lds_fence();
            const Key x = i + lane < n ? lds.got[i + lane] : 0;
            const bool in = x >= least && x > last;
            const uint64_t mask = __ballot(in);
            wave_lds_fence();
            if (in)
                lds.got[left + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                              __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0))] = x;
            left += __popcll(mask);
        }
        wave_lds_fence();
        for (int i = 0; i < left;) {
            const int have = __ballot(lane < k && key != 0) ? k : 0;  // entries of the list
            const int more = min(left - i, 64 - have);
            Key x = lane < have ? key : 0;
            if (lane >= have && lane < have + more)
                x = lds.got[i + lane - have];
            i += more;
            if (!__ballot(lane >= have && x > last))
                continue;
            int rank = 0;
            for (int j = 0; j < have + more; ++j)
                rank += lane_key(x, j) > x ? 1 : 0;
            if (lane < k)
                lds.list[lane] = 0;
            wave_lds_fence();
            if (x != 0 && rank < k)
                lds.list[rank] = x;
            wave_lds_fence();
            key = lane < k ? lds.list[lane] : 0;
            wave_lds_fence();
            last = lane_key(key, k - 1);
        }
    }
};

// k-th largest of the lanes' values (k <= 64) or less, -inf if it is not finite: bit after
// bit of the largest bound that k lanes reach
__device__ __forceinline__ float kth_of_lanes(float x, int k)
{
    const uint32_t key = order_of(x);
    uint32_t bound = 0;
    for (int bit = 31; bit >= 16; --bit) {  // the low bits are left at 0: still a bound from below
        const uint32_t next = bound | (1u << bit);
        if (__popcll(__ballot(key >= next)) >= k)
            bound = next;
    }
    const float f = of_order(bound);
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
            } else if (i + VE <= left) {
                // 16 bytes at an element's alignment: global memory takes them in one access
                typedef u32x4 Unaligned __attribute__((aligned(2)));
                w[l] = *reinterpret_cast<const Unaligned *>(p + i);
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
                          Top &top, TopLds &lds, uint32_t &reached)
{
    using Tile = LogitTile<T>;
    sums = {neg_inf(), 0.0f, 0.0f};
    top.key = top.last = 0;
    constexpr int N = 64 * kTile;
    Tile next;
    if (begin < end)
        next.template load<VEC>(row + begin, end - begin, lane);
    float most = neg_inf();   // of the lane, over all tiles
    float bound = neg_inf();  // at least k logits reach it
    // above a full list's last entry: an equal logit of a later tile comes behind it
    float above = neg_inf();
    int n = 0;                // candidates gathered
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
        // the best bound of the workgroup's waves: k logits of the row reach it
        const uint32_t others = __hip_atomic_load(&reached, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
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
        if (k > 0)
            bound = fmaxf(bound, of_order(others));
        if (k > 0 && __ballot(m >= fmaxf(bound, above))) {
            most = fmaxf(most, m);
            bound = fmaxf(bound, kth_of_lanes(most, k));
            if (lane == 0)
                __hip_atomic_fetch_max(&reached, order_of(bound), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            if (n > kGather) {
                top.take(lds, n, bound, k, lane);
                n = 0;
                above = top.last ? next_above(logit_of(top.last)) : neg_inf();
            }
            const float least = fmaxf(bound, above);
#pragma unroll
            for (int l = 0; l < Tile::NL; ++l)
#pragma unroll
                for (int e = 0; e < Tile::VE; ++e) {
                    const float v = x[l * Tile::VE + e];
                    const bool may = v >= least;
                    if (__ballot(may)) {
                        const int at = Tile::at(lane, l, e);
                        // of what a mask left out only the first k logits count: nothing is
                        // below it, and they come first
                        const bool in = may && at < left && (v > neg_inf() || (base == begin && at < k));
                        const uint64_t mask = __ballot(in);
                        if (in)
                            lds.got[n + (int)__builtin_amdgcn_mbcnt_hi(
                                            (uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0))] =
                                key_of(v, (int)base + at);
                        n += __popcll(mask);
                    }
                }
        }
    }
    if (n > 0)
        top.take(lds, n, bound, k, lane);
    sums = wave_join(sums);
}

__device__ __forceinline__ bool row_live(const LogprobParams &p, int row)
{
    const int b = row / p.num_tokens, t = row - b * p.num_tokens;
    return (!p.idx || p.idx[b] >= 0) && (!p.ctx || t < p.ctx[b]);
}

// The given token's logit, read early
struct Given {
    float x;
    bool outside;  // of [0, V)
};
template <typename T>
__device__ __forceinline__ Given given_logit(const LogprobParams &p, int row, const T *logits)
{
    const int tok = p.tokens[row];
    Given g = {0.0f, tok < 0 || tok >= p.vocab};
    if (!g.outside)
        g.x = ld_elem<T>(logits, tok);
    return g;
}

// The answers of a row from its sums; lane i < k holds entry i of the list.
__device__ void write_row(const LogprobParams &p, int64_t row, const Given &given, const Sums &a,
                          Key key, int lane)
{
    const float nan = __builtin_nanf("");
    const float log_s = logf(a.s);
    const bool bad = a.s != a.s;
    // x - lse as (x - m) - log s: exact differences of large logits first
    auto logprob = [&](float x) {
        return bad ? nan : x == neg_inf() ? neg_inf() : (x - a.m) - log_s;
    };
    if (lane == 0) {
        p.logprobs[row] = given.outside ? neg_inf() : logprob(given.x);
        if (p.entropy)
            p.entropy[row] = bad ? nan : a.m == neg_inf() ? 0.0f : fmaxf(log_s - a.t / a.s, 0.0f);
    }
    if (lane < p.top) {
        const bool none = key == 0;  // only beside NaN
        p.top_ids[row * p.top + lane] = none ? -1 : index_of(key);
        p.top_logprobs[row * p.top + lane] = none ? nan : logprob(logit_of(key));
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

// The k best of `parts` ordered lists of k keys. The best of the lists' last entries bounds
// them from below; the few that reach it are gathered, and each one's place is the number
// of better ones.
struct Gathered {
    unsigned long long bound;
    int n;
};

__device__ void place_lists(const Key *lists, int parts, int k, Key *got, Gathered &g, Key *out)
{
    if (threadIdx.x == 0)
        g = {0, 0};
    for (int i = threadIdx.x; i < k; i += blockDim.x)
        out[i] = 0;
    __syncthreads();
    if ((int)threadIdx.x < parts)
        atomicMax(&g.bound, (unsigned long long)lists[threadIdx.x * k + k - 1]);
    __syncthreads();
    const Key bound = g.bound;
    for (int i = threadIdx.x; i < parts * k; i += blockDim.x) {
        const Key x = lists[i];
        if (x != 0 && x >= bound)
            got[atomicAdd(&g.n, 1)] = x;  // in any order: places come from the values
    }
    __syncthreads();
    const int m = g.n;
    for (int i = threadIdx.x; i < m; i += blockDim.x) {
        const Key x = got[i];
        int at = 0;
#pragma unroll 8
        for (int j = 0; j < m; ++j)
            at += got[j] > x ? 1 : 0;
        if (at < k)
            out[at] = x;
    }
    __syncthreads();
}

// Part of a row in the workspace: its sums (and a word for the alignment), then k keys.
__host__ __device__ inline int64_t part_words(int64_t top) { return 4 + 2 * top; }

template <typename T, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void logprobs_kernel(LogprobParams p, int parts, int part, int row0)
{
    __shared__ Sums sums_of[kWaves];
    __shared__ Key lists[kWaves * kMaxTop], best[kMaxTop];
    __shared__ TopLds tops[kWaves];
    __shared__ Gathered gathered;
    __shared__ uint32_t reached;  // a bound's order_of; 0 is that of a NaN, which bounds nothing
    if (threadIdx.x == 0)
        reached = 0;
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int which = (int)(blockIdx.x % (uint32_t)parts);
    const int row = row0 + (int)(blockIdx.x / (uint32_t)parts);
    if (!row_live(p, row)) {
        if (which == 0 && wave == 0)
            write_padding(p, row, lane);
        return;
    }
    const int b = row / p.num_tokens, t = row - b * p.num_tokens;
    const T *logits = static_cast<const T *>(p.logits) + b * p.l_bs + t * p.l_rs;
    Given given = {};
    if (parts == 1 && wave == 0)
        given = given_logit<T>(p, row, logits);
    const int64_t begin = (int64_t)which * part;
    const int end = (int)min((int64_t)p.vocab, begin + part);
    Sums sums;
    Top top;
    const int64_t mine = begin + (int64_t)wave * 64 * kTile;
    wave_pass<T, VEC>(logits, (int)min(mine, (int64_t)end), end, kWaves, p.top, lane, sums, top,
                      tops[wave], reached);
    if (lane == 0)
        sums_of[wave] = sums;
    if (lane < p.top)
        lists[wave * p.top + lane] = top.key;
    __syncthreads();
    if (p.top > 0)
        place_lists(lists, kWaves, p.top, tops[0].got, gathered, best);
    if (wave != 0)
        return;
    Sums a = sums_of[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
        a = join(a, sums_of[w]);
    const Key key = lane < p.top ? best[lane] : 0;
    if (parts == 1) {
        write_row(p, row, given, a, key, lane);
        return;
    }
    float *w = static_cast<float *>(p.workspace) + ((int64_t)row * parts + which) * part_words(p.top);
    if (lane == 0)
        *reinterpret_cast<Sums *>(w) = a;
    if (lane < p.top)
        reinterpret_cast<Key *>(w + 4)[lane] = key;
}

constexpr int kMaxParts = 64;

template <typename T>
__global__ __launch_bounds__(256) void logprobs_join_kernel(LogprobParams p, int parts)
{
    __shared__ Key lists[kMaxParts * kMaxTop], got[kMaxParts * kMaxTop], best[kMaxTop];
    __shared__ Gathered gathered;
    const int lane = threadIdx.x & 63;
    const int row = blockIdx.x;
    if (!row_live(p, row))
        return;
    const int b = row / p.num_tokens, t = row - b * p.num_tokens;
    const T *logits = static_cast<const T *>(p.logits) + b * p.l_bs + t * p.l_rs;
    const int64_t pw = part_words(p.top);
    const float *w = static_cast<const float *>(p.workspace) + (int64_t)row * parts * pw;
    const bool first = threadIdx.x < 64;
    Given given = {};
    Sums a = {neg_inf(), 0.0f, 0.0f};
    if (first) {  // in flight with the lists
        given = given_logit<T>(p, row, logits);
        if (lane < parts)
            a = *reinterpret_cast<const Sums *>(w + lane * pw);
    }
    for (int i = threadIdx.x; i < parts * p.top; i += blockDim.x) {
        const int q = i / p.top, j = i - q * p.top;
        lists[i] = reinterpret_cast<const Key *>(w + q * pw + 4)[j];
    }
    __syncthreads();
    if (p.top > 0)
        place_lists(lists, parts, p.top, got, gathered, best);
    if (!first)
        return;
    a = wave_join(a);
    write_row(p, row, given, a, lane < p.top ? best[lane] : 0, lane);
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
    const int64_t e = sizeof(T);
    const bool vec = ((uintptr_t)p.logits | (uintptr_t)(p.l_bs * e) | (uintptr_t)(p.l_rs * e)) % 16 == 0;
    // a launch has fewer than 2^32 threads; rows of several parts are few
    constexpr int64_t kRows = 1 << 23;
    for (int64_t row0 = 0; row0 < rows; row0 += kRows) {
        const int64_t some = rows - row0 < kRows ? rows - row0 : kRows;
        if (!launchable((__int128)some * parts, 64 * kWaves))
            return hipErrorInvalidConfiguration;
        const dim3 grid((uint32_t)(some * parts));
        if (vec)
            logprobs_kernel<T, true><<<grid, 64 * kWaves, 0, stream>>>(p, parts, part, (int)row0);
        else
            logprobs_kernel<T, false><<<grid, 64 * kWaves, 0, stream>>>(p, parts, part, (int)row0);
    }
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
