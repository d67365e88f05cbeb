// Verification of drafted tokens against the target's probabilities from given
// random numbers, and the draw of the token after them.
//
// Which tokens stand needs one entry of p (and q) per token: a wave gathers
// them, one or two tokens a lane, and walks the path with ballots. The token
// after them is drawn by inverting the distribution function of one row of
// weights: fp64 sums of segments of 512 vocabulary entries (a wave each, eight
// adjacent entries a lane), then one wave finds the first segment whose running
// sum passes u times the total, and the entry in it. Every sum has a fixed
// order. Long rows take two launches, with the segments spread over the GPU;
// rows that one workgroup reads as fast as a second launch costs take one.
// The row is read once, so HBM bounds large vocabularies; a small one is a
// chain of dependent accesses (lengths, tokens, gathered entries, the row, a
// segment again).
// Measured: 64 x 131072 fp32 with draft probabilities 14.3-14.9 us for the sums (4.5
// TB/s) and 4.1-4.7 for the draw; 16 trees of 64 nodes x 32000 bf16 10.4. One launch |
// two, fp32: 64 x 32000 11.2 | 13.9 us, 1 x 32000 9.0 | 9.0, 1 x 2000 8.1 | 9.6.
#include "ssu_device.h"
#include "ssu_internal.h"

namespace ssu {
namespace {

constexpr int kPer = 8;  // adjacent entries of a lane
constexpr int kNodes = SSU_MAX_TREE_NODES;
static_assert(kVerifySegment == 64 * kPer, "a segment is a wave's load");

// What the walk leaves: accepted tokens, the last accepted one, whether the
// weights subtract the draft's row, the path, and the rejected children.
struct Walk {
    int count, last, subtract, removed_n, tried;
    int path[kNodes];
    int removed[kNodes];
};

// The tokens of node at's children (lane i holds nodes i and i + 64), in `to`;
// returns how many.
__device__ __forceinline__ int list_children(const int (&par)[2], const int (&tok)[2], int at, int *to)
{
    int n = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const uint64_t kids = __ballot(par[s] == at);
        if (par[s] == at)
            to[n + __popcll(kids & ((1ull << (threadIdx.x & 63)) - 1))] = tok[s];
        n += __popcll(kids);
    }
    return n;
}

__device__ __forceinline__ double bcast(double v, int lane)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// v of the lanes that CTRL shifts from, 0 where there is none or the row is
// masked off.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, false);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Inclusive sums over the wave's lanes: within rows of 16, then lane 15 to the
// odd rows, then lane 31 to the upper half.
__device__ __forceinline__ double wave_scan(double v)
{
    v += dpp_f64<0x111, 0xF>(v);  // row_shr:1
    v += dpp_f64<0x112, 0xF>(v);  // row_shr:2
    v += dpp_f64<0x114, 0xF>(v);  // row_shr:4
    v += dpp_f64<0x118, 0xF>(v);  // row_shr:8
    v += dpp_f64<0x142, 0xA>(v);  // row_bcast:15
    v += dpp_f64<0x143, 0xC>(v);  // row_bcast:31
    return v;
}
__device__ __forceinline__ double wave_total(double v) { return bcast(wave_scan(v), 63); }

// The walk of row b by one wave (all 64 lanes); lane i holds nodes i and i+64.
template <typename T>
__device__ __forceinline__ void walk_row(const VerifyParams &p, int b, int len, Walk &w)
{
    const int lane = threadIdx.x & 63;
    const int n = p.num_tokens;
    int par[2], tok[2];
    double prob[2], u[2], q[2];
    // the row's tokens are loaded whole, beside its length, and masked after
    float uf[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int64_t i = (int64_t)b * n + min(lane + 64 * s, n - 1);
        tok[s] = p.tokens[i];
        par[s] = p.parents ? p.parents[i] : lane + 64 * s - 1;
        uf[s] = p.uniforms[i];
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int m = lane + 64 * s;
        const bool in = m >= 1 && m < len;
        tok[s] = in ? tok[s] : -1;
        par[s] = in ? par[s] : -1;
        u[s] = in ? (double)uf[s] : 0.0;
        if (par[s] < 0 || par[s] >= m)
            par[s] = -1;
        const bool ok = par[s] >= 0 && tok[s] >= 0 && tok[s] < p.vocab;
        prob[s] = ok ? (double)ld_elem<T>(p.target, b * p.t_bs + par[s] * p.t_rs + tok[s])
                     : 0.0;
        q[s] = ok && p.draft
                   ? (double)ld_elem<T>(p.draft, b * p.d_bs + (m - 1) * p.d_rs + tok[s])
                   : 0.0;
        if (!(prob[s] > 0.0))  // negative and NaN count as no probability
            prob[s] = 0.0;
    }
    int count = 1, last = 0, subtract = 0, removed_n = 0;
    if (lane == 0)
        w.path[0] = 0;
    if (p.draft) {
        // accepted up to the first rejected token
        uint64_t rej[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int m = lane + 64 * s;
            rej[s] = __ballot(m >= 1 && m < len && !(u[s] * q[s] < prob[s]));
        }
        int first = rej[0] ? __ffsll((unsigned long long)rej[0]) - 1
                           : (rej[1] ? 63 + __ffsll((unsigned long long)rej[1]) : len);
        count = min(first, p.max_accept);
        last = count - 1;
        // after max_accept tokens none was rejected: the target's row itself
        subtract = first < len && first < p.max_accept;
        for (int m = lane; m < count; m += 64)
            w.path[m] = m;
    } else {
        // A node's children are tried all at once: child c stands if u (1 - the
        // p of the children before it) < p, and the first that stands is taken.
        int at = 0;
        while (count < p.max_accept) {
            uint64_t kids[2], stand[2];
#pragma unroll
            for (int s = 0; s < 2; ++s)
                kids[s] = __ballot(par[s] == at);
            if (!(kids[0] | kids[1]))
                break;
            // of a token that a sibling has before, nothing is left
            double left[2] = {prob[0], prob[1]};
            for (uint64_t k0 = kids[0], k1 = kids[1]; (k0 & (k0 - 1)) | k1;) {
                const int c = k0 ? 0 : 1, l = __ffsll((unsigned long long)(k0 ? k0 : k1)) - 1;
                k0 &= k0 - 1;  // 0 stays 0
                if (c)
                    k1 &= k1 - 1;
                const int x = __builtin_amdgcn_readlane(c ? tok[1] : tok[0], l), m = l + 64 * c;
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    left[s] = par[s] == at && tok[s] == x && lane + 64 * s > m ? 0.0 : left[s];
            }
            double before = 0.0;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const double mine = par[s] == at ? left[s] : 0.0;
                double sum = 0.0;
                if (kids[s] & (kids[s] - 1))  // more than one
                    sum = wave_scan(mine);
                else
                    sum = mine;
                stand[s] = __ballot(par[s] == at && u[s] * (1.0 - (before + (sum - mine))) < mine);
                if (s == 0 && kids[0])
                    before = kids[0] & (kids[0] - 1)
                                 ? bcast(sum, 63)
                                 : bcast(mine, __ffsll((unsigned long long)kids[0]) - 1);
            }
            if (!(stand[0] | stand[1]))
                break;
            at = stand[0] ? __ffsll((unsigned long long)stand[0]) - 1
                          : 63 + __ffsll((unsigned long long)stand[1]);
            if (lane == 0)
                w.path[count] = at;
            ++count;
        }
        removed_n = count < p.max_accept ? list_children(par, tok, at, w.removed) : 0;
        last = at;
    }
    if (lane == 0) {
        w.count = count;
        w.last = last;
        w.subtract = subtract;
        w.tried = count < p.max_accept;
        w.removed_n = removed_n;
    }
}

// The row of weights that is drawn from.
struct Row {
    const void *p, *q;  // q null: the target's row alone
    const int *removed;
    int removed_n, vocab;
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const void *p, int64_t i, int n, float (&v)[kPer])
{
    if constexpr (VEC) {
        if (n >= kPer) {
            ld_typed<T, kPer>(p, i, v);
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        v[j] = j < n ? ld_elem<T>(p, i + j) : 0.0f;
}

// The weights of the lane's entries of a segment: the target's row, less the
// draft's; 0 for removed entries, entries past the vocabulary, and negative or
// NaN weights.
template <typename T, bool VEC>
__device__ __forceinline__ void weights8(const Row &r, int segment, double (&w)[kPer])
{
    const int v0 = segment * kVerifySegment + (int)(threadIdx.x & 63) * kPer;
    const int n = r.vocab - v0;
    float p[kPer], q[kPer];
    load8<T, VEC>(r.p, v0, n, p);
    if (r.q)
        load8<T, VEC>(r.q, v0, n, q);
    uint32_t gone = 0;
    for (int k = 0; k < r.removed_n; ++k) {
        const unsigned at = (unsigned)(r.removed[k] - v0);
        gone |= at < (unsigned)kPer ? 1u << at : 0u;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const double x = r.q ? (double)p[j] - (double)q[j] : (double)p[j];
        w[j] = x > 0.0 && !((gone >> j) & 1u) ? x : 0.0;
    }
}

__device__ __forceinline__ double sum8(const double (&w)[kPer])
{
    return ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
}

// Sums of segments k0, k0 + step, .. below `end`, by one wave, U loaded together.
template <typename T, bool VEC, int U>
__device__ __forceinline__ void sum_segments(const Row &r, int k0, int step, int end, double *sums)
{
    for (int k = k0; k < end; k += U * step) {
        double t[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            double e[kPer];
            weights8<T, VEC>(r, min(k + i * step, end - 1), e);
            t[i] = sum8(e);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            t[i] = wave_total(t[i]);
            if ((threadIdx.x & 63) == 0 && k + i * step < end)
                sums[k + i * step] = t[i];
        }
    }
}

// Draws from the row given its segments' sums, by one wave. -1 without mass.
template <typename T, bool VEC>
__device__ int draw(const Row &r, const double *sums, int segments, double u)
{
    const int lane = threadIdx.x & 63;
    // a lane has a run of segments
    const int run = (segments + 63) / 64;
    const int s0 = min(lane * run, segments), s1 = min(s0 + run, segments);
    double own = 0.0;
    for (int k = s0; k < s1; ++k)
        own += sums[k];
    const double incl = wave_scan(own);
    const double total = bcast(incl, 63);
    if (!(total > 0.0))
        return -1;
    const double goal = u * total;
    const uint64_t some = __ballot(own > 0.0), hit = __ballot(own > 0.0 && incl > goal);
    // nothing passes (the goal rounds up to the total): the last entry with mass
    const bool over = hit == 0;
    const int l = over ? 63 - __clzll((unsigned long long)some) : __ffsll((unsigned long long)hit) - 1;
    // the segment in lane l's run
    double before = 0.0;
    int segment = 0;
    if (lane == l) {
        before = incl - own;
        int last = s0;
        double at = before, last_before = before;
        bool found = false;
        for (int k = s0; k < s1 && !found; ++k) {
            const double s = sums[k];
            if (s > 0.0) {
                last = k, last_before = at;
                found = !over && at + s > goal;
            }
            at += s;
        }
        segment = last;
        before = last_before;
    }
    segment = __builtin_amdgcn_readlane(segment, l);
    before = bcast(before, l);
    // the entry in the segment
    double w[kPer];
    weights8<T, VEC>(r, segment, w);
    const double sum = sum8(w), in = wave_scan(sum);
    double at = before + (in - sum);
    const int v0 = segment * kVerifySegment + lane * kPer;
    int first = -1, last = -1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        at += w[j];
        if (w[j] > 0.0) {
            last = v0 + j;
            if (first < 0 && !over && at > goal)
                first = last;
        }
    }
    const uint64_t firsts = __ballot(first >= 0), lasts = __ballot(last >= 0);
    if (firsts)
        return __builtin_amdgcn_readlane(first, __ffsll((unsigned long long)firsts) - 1);
    return __builtin_amdgcn_readlane(last, 63 - __clzll((unsigned long long)lasts));
}

// The same with the target's own row where the weights had no mass.
template <typename T, bool VEC>
__device__ int draw_or_target(Row r, double *sums, int segments, double u)
{
    int v = draw<T, VEC>(r, sums, segments, u);
    if (v >= 0 || (!r.q && r.removed_n == 0))
        return v;
    r.q = nullptr;
    r.removed_n = 0;
    __threadfence_block();  // this wave's reads of sums are done before it rewrites them
    sum_segments<T, VEC, 1>(r, 0, 1, segments, sums);
    __threadfence_block();
    return draw<T, VEC>(r, sums, segments, u);
}

__device__ __forceinline__ int row_length(const VerifyParams &p, int b)
{
    if (p.idx && p.idx[b] < 0)
        return 0;
    return p.ctx ? clamp_len(p.ctx[b], p.num_tokens) : p.num_tokens;
}

template <typename T>
__device__ __forceinline__ Row row_of(const VerifyParams &p, int b, const Walk &w)
{
    constexpr int ES = sizeof(T) == 4 ? 4 : 2;
    Row r;
    r.p = static_cast<const char *>(p.target) + (b * p.t_bs + w.last * p.t_rs) * ES;
    r.q = w.subtract ? static_cast<const char *>(p.draft) + (b * p.d_bs + w.last * p.d_rs) * ES
                     : nullptr;
    r.removed = w.removed;
    r.removed_n = w.removed_n;
    r.vocab = p.vocab;
    return r;
}

// accepted_lengths and the path, by the workgroup that walked.
__device__ __forceinline__ void write_path(const VerifyParams &p, int b, int len, const Walk &w)
{
    const int count = len > 0 ? w.count : 0;
    if (threadIdx.x == 0)
        p.accepted[b] = count;
    if (p.path)
        for (int i = threadIdx.x; i < p.max_accept; i += blockDim.x)
            p.path[(int64_t)b * p.max_accept + i] = i < count ? w.path[i] : -1;
}

// One launch: a workgroup a row.
template <typename T, bool VEC>
__global__ __launch_bounds__(1024) void ssu_verify_row_kernel(const VerifyParams p, int segments)
{
    __shared__ Walk w;
    __shared__ double sums[kVerifyRowSegments];
    const int b = blockIdx.x;
    const int len = row_length(p, b);
    const double u = (double)p.uniforms[(int64_t)b * p.num_tokens];
    if (threadIdx.x < 64)
        walk_row<T>(p, b, len, w);
    __syncthreads();
    write_path(p, b, len, w);
    if (len == 0) {
        if (threadIdx.x == 0)
            p.next[b] = -1;
        return;
    }
    const Row r = row_of<T>(p, b, w);
    sum_segments<T, VEC, 4>(r, threadIdx.x >> 6, 16, segments, sums);
    __syncthreads();
    if (threadIdx.x < 64) {
        const int v = draw_or_target<T, VEC>(r, sums, segments, u);
        if (threadIdx.x == 0)
            p.next[b] = v;
    }
}

// Two launches: the sums, `each` segments a wave, by workgroups that all walk
// (the walk is short beside the row) ..
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void ssu_verify_sums_kernel(const VerifyParams p, int segments,
                                                              int each)
{
    __shared__ Walk w;
    const int b = blockIdx.y;
    const int len = row_length(p, b);
    if (threadIdx.x < 64)
        walk_row<T>(p, b, len, w);
    __syncthreads();
    if (blockIdx.x == 0)
        write_path(p, b, len, w);
    if (len == 0)
        return;
    const Row r = row_of<T>(p, b, w);
    double *sums = p.partial + (int64_t)b * (segments + 1);
    if (blockIdx.x == 0 && threadIdx.x == 0)  // for the draw
        reinterpret_cast<uint64_t *>(sums)[segments] = w.last | (w.subtract ? 256 : 0) | (w.tried ? 512 : 0);
    const int k0 = (blockIdx.x * 4 + (int)(threadIdx.x >> 6)) * each;
    sum_segments<T, VEC, 1>(r, k0, 1, min(k0 + each, segments), sums);
}

// .. and the draw, a wave a row.
template <typename T, bool VEC>
__global__ __launch_bounds__(64) void ssu_verify_draw_kernel(const VerifyParams p, int segments)
{
    __shared__ Walk w;
    const int b = blockIdx.x;
    const int len = row_length(p, b);
    if (len == 0) {
        if (threadIdx.x == 0)
            p.next[b] = -1;
        return;
    }
    double *sums = p.partial + (int64_t)b * (segments + 1);
    const uint64_t word = reinterpret_cast<const uint64_t *>(sums)[segments];
    const int last = (int)(word & 255);
    int par[2], tok[2], removed_n = 0;
    if (!p.draft) {  // the last node's children, if they were tried, were all rejected
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int m = threadIdx.x + 64 * s;
            const bool in = m >= 1 && m < len;
            const int64_t i = (int64_t)b * p.num_tokens + m;
            tok[s] = in ? p.tokens[i] : -1;
            par[s] = in ? (p.parents ? p.parents[i] : m - 1) : -1;
            if (par[s] >= m)
                par[s] = -1;
        }
        if (word & 512)
            removed_n = list_children(par, tok, last, w.removed);
    }
    if (threadIdx.x == 0) {
        w.last = last;
        w.subtract = (word & 256) != 0;
        w.removed_n = removed_n;
    }
    __syncthreads();
    const Row r = row_of<T>(p, b, w);
    const int v = draw_or_target<T, VEC>(r, sums, segments,
                                         (double)p.uniforms[(int64_t)b * p.num_tokens]);
    if (threadIdx.x == 0)
        p.next[b] = v;
}

template <typename T, bool VEC>
hipError_t launch_verify_type(const VerifyParams &p, hipStream_t stream)
{
    const int segments = (p.vocab + kVerifySegment - 1) / kVerifySegment;
    if (segments <= kVerifyRowSegments) {
        hipLaunchKernelGGL((ssu_verify_row_kernel<T, VEC>), dim3((unsigned)p.batch), dim3(1024), 0,
                           stream, p, segments);
        return hipGetLastError();
    }
    int each = (int)(((int64_t)segments * p.batch + 1024 * 4 - 1) / (1024 * 4));
    each = each < 1 ? 1 : each > 16 ? 16 : each;
    const int blocks = (segments + 4 * each - 1) / (4 * each);
    hipLaunchKernelGGL((ssu_verify_sums_kernel<T, VEC>), dim3((unsigned)blocks, (unsigned)p.batch),
                       dim3(256), 0, stream, p, segments, each);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((ssu_verify_draw_kernel<T, VEC>), dim3((unsigned)p.batch), dim3(64), 0, stream,
                       p, segments);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_verify_rows(const VerifyParams &p, hipStream_t stream)
{
    constexpr int ES = sizeof(T) == 4 ? 4 : 2, PER = 16 / ES;
    const bool vec = (uintptr_t)p.target % 16 == 0 && p.t_bs % PER == 0 && p.t_rs % PER == 0 &&
                     (uintptr_t)p.draft % 16 == 0 && p.d_bs % PER == 0 && p.d_rs % PER == 0;
    return vec ? launch_verify_type<T, true>(p, stream) : launch_verify_type<T, false>(p, stream);
}

}  // namespace

hipError_t launch_verify(const VerifyParams &p, hipStream_t stream)
{
    (void)hipGetLastError();  // report only this launch's status
    switch (p.prob_dtype) {
    case kF32: return launch_verify_rows<float>(p, stream);
    case kF16: return launch_verify_rows<_Float16>(p, stream);
    default: return launch_verify_rows<bf16_t>(p, stream);
    }
}

}  // namespace ssu
