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
    int count, last, subtract, removed_n;
    int path[kNodes];
    int removed[kNodes];
};

__device__ __forceinline__ double bcast(double v, int lane)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// The walk of row b by one wave (all 64 lanes); lane i holds nodes i and i+64.
template <typename T>
__device__ __forceinline__ void walk_row(const VerifyParams &p, int b, int len, Walk &w)
{
    const int lane = threadIdx.x & 63;
    const int n = p.num_tokens;
    int par[2], tok[2];
    double prob[2], u[2], q[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int m = lane + 64 * s;
        const bool in = m >= 1 && m < len;
        tok[s] = in ? p.tokens[(int64_t)b * n + m] : -1;
        par[s] = in ? (p.parents ? p.parents[(int64_t)b * n + m] : m - 1) : -1;
        u[s] = in ? (double)p.uniforms[(int64_t)b * n + m] : 0.0;
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
        int at = 0;
        double left = 1.0;
        uint64_t kids[2];
        auto children = [&]() {
#pragma unroll
            for (int s = 0; s < 2; ++s)
                kids[s] = __ballot(par[s] == at);
        };
        children();
        while (count < p.max_accept && (kids[0] | kids[1])) {
            const int s = kids[0] ? 0 : 1;
            const int l = __ffsll((unsigned long long)kids[s]) - 1;
            kids[s] &= kids[s] - 1;
            const int x = __builtin_amdgcn_readlane(s ? tok[1] : tok[0], l);
            const int m = l + 64 * s;
            const double uc = bcast(s ? u[1] : u[0], l);
            double pc = bcast(s ? prob[1] : prob[0], l);
            // a sibling before it had the same token: nothing of it is left
            const uint64_t again0 = __ballot(par[0] == at && tok[0] == x && lane < m);
            const uint64_t again1 = __ballot(par[1] == at && tok[1] == x && lane + 64 < m);
            if (again0 | again1)
                pc = 0.0;
            if (uc * left < pc) {
                if (lane == 0)
                    w.path[count] = m;
                ++count;
                at = m;
                left = 1.0;
                removed_n = 0;
                children();
            } else {
                left -= pc;
                if (lane == 0)
                    w.removed[removed_n] = x;
                ++removed_n;
            }
        }
        last = at;
    }
    if (lane == 0) {
        w.count = count;
        w.last = last;
        w.subtract = subtract;
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

// Inclusive sums over the wave's lanes.
__device__ __forceinline__ double wave_scan(double v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_up(v, m, 64);
        if (lane >= m)
            v += o;
    }
    return v;
}
__device__ __forceinline__ double wave_total(double v)
{
#pragma unroll
    for (int m = 32; m > 0; m >>= 1)
        v += __shfl_xor(v, m, 64);
    return v;
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
    for (int k = 0; k < segments; ++k) {
        double w[kPer];
        weights8<T, VEC>(r, k, w);
        const double t = wave_total(sum8(w));
        if ((threadIdx.x & 63) == 0)
            sums[k] = t;
    }
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
    if (len > 0 && threadIdx.x < 64)
        walk_row<T>(p, b, len, w);
    __syncthreads();
    write_path(p, b, len, w);
    if (len == 0) {
        if (threadIdx.x == 0)
            p.next[b] = -1;
        return;
    }
    const Row r = row_of<T>(p, b, w);
    for (int k = threadIdx.x >> 6; k < segments; k += 16) {
        double e[kPer];
        weights8<T, VEC>(r, k, e);
        const double t = wave_total(sum8(e));
        if ((threadIdx.x & 63) == 0)
            sums[k] = t;
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        const int v = draw_or_target<T, VEC>(r, sums, segments,
                                             (double)p.uniforms[(int64_t)b * p.num_tokens]);
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
    if (len > 0 && threadIdx.x < 64)
        walk_row<T>(p, b, len, w);
    __syncthreads();
    if (blockIdx.x == 0)
        write_path(p, b, len, w);
    if (len == 0)
        return;
    const Row r = row_of<T>(p, b, w);
    double *sums = p.partial + (int64_t)b * (segments + 1);
    const int k0 = (blockIdx.x * 4 + (int)(threadIdx.x >> 6)) * each;
    for (int k = k0; k < min(k0 + each, segments); ++k) {
        double e[kPer];
        weights8<T, VEC>(r, k, e);
        const double t = wave_total(sum8(e));
        if ((threadIdx.x & 63) == 0)
            sums[k] = t;
    }
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
    walk_row<T>(p, b, len, w);
    __syncthreads();
    const Row r = row_of<T>(p, b, w);
    const int v = draw_or_target<T, VEC>(r, p.partial + (int64_t)b * (segments + 1), segments,
                                         (double)p.uniforms[(int64_t)b * p.num_tokens]);
    if (threadIdx.x == 0)
        p.next[b] = v;
}

template <typename T, bool VEC>
hipError_t launch_verify_type(const VerifyParams &p, hipStream_t stream)
{
    const int segments = (p.vocab + kVerifySegment - 1) / kVerifySegment;
#ifndef ROWSEG
#define ROWSEG kVerifyRowSegments
#endif
    if (segments <= ROWSEG) {
        hipLaunchKernelGGL((ssu_verify_row_kernel<T, VEC>), dim3((unsigned)p.batch), dim3(1024), 0,
                           stream, p, segments);
        return hipGetLastError();
    }
#ifndef VWG
#define VWG 2048
#endif
    int each = (int)(((int64_t)segments * p.batch + VWG * 4 - 1) / (VWG * 4));
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
