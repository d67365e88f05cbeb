// Verification of drafted tokens against the target's probabilities from given
// random numbers, and the draw of the token after them.
//
// Which tokens stand needs one entry of p (and q) per token: a wave gathers
// them, one or two tokens a lane, and walks the path with ballots. The token
// after them is drawn by inverting the distribution function of one row of
// weights: fp64 sums over chunks of kVerifyChunk vocabulary entries (first
// launch, one workgroup a chunk), then (second launch, one workgroup a row)
// the first chunk whose running sum passes u times the total, and the entry in
// it. Every sum has a fixed order.
#include "ssu_device.h"
#include "ssu_internal.h"

namespace ssu {
namespace {

constexpr int kNT = 256;
constexpr int kPer = kVerifyChunk / kNT;  // consecutive entries per thread
constexpr int kNodes = SSU_MAX_TREE_NODES;
static_assert(kPer == 8, "a thread's entries are one byte of the removed-token bitmap");

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
__device__ void walk_row(const VerifyParams &p, int b, int len, Walk &w)
{
    const int lane = threadIdx.x & 63;
    const int T = p.num_tokens;
    int par[2], tok[2];
    double prob[2], u[2], q[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int m = lane + 64 * s;
        const bool in = m >= 1 && m < len;
        tok[s] = in ? p.tokens[(int64_t)b * T + m] : -1;
        par[s] = in ? (p.parents ? p.parents[(int64_t)b * T + m] : m - 1) : -1;
        u[s] = in ? (double)p.uniforms[(int64_t)b * T + m] : 0.0;
        if (par[s] < 0 || par[s] >= m)
            par[s] = -1;
        const bool ok = par[s] >= 0 && tok[s] >= 0 && tok[s] < p.vocab;
        prob[s] = ok ? (double)ld_io(p.target, b * p.t_bs + par[s] * p.t_rs + tok[s], p.prob_dtype)
                     : 0.0;
        q[s] = ok && p.draft
                   ? (double)ld_io(p.draft, b * p.d_bs + (m - 1) * p.d_rs + tok[s], p.prob_dtype)
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

// The weights of entries v0 .. v0+7: the target's row, less the draft's where
// `sub`; `gone` has a bit per removed entry. Entries past the vocabulary, and
// negative or NaN weights, are 0.
__device__ __forceinline__ void weights8(const VerifyParams &p, int64_t t_off, int64_t d_off,
                                         int v0, bool sub, uint32_t gone, double (&w)[kPer])
{
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        double x = 0.0;
        if (v0 + j < p.vocab) {
            x = (double)ld_io(p.target, t_off + v0 + j, p.prob_dtype);
            if (sub)
                x -= (double)ld_io(p.draft, d_off + v0 + j, p.prob_dtype);
        }
        w[j] = x > 0.0 && !((gone >> j) & 1u) ? x : 0.0;
    }
}

// Bits of the chunk's removed entries: byte t of `bits` belongs to thread t.
__device__ __forceinline__ uint32_t removed_bits(const Walk &w, int base, uint32_t *bits)
{
    if (w.removed_n == 0)
        return 0;
    if (threadIdx.x < kNT / 4)
        bits[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < w.removed_n; i += kNT) {
        const unsigned k = (unsigned)(w.removed[i] - base);
        if (k < (unsigned)kVerifyChunk)
            atomicOr(&bits[k >> 5], 1u << (k & 31));
    }
    __syncthreads();
    return (bits[threadIdx.x >> 2] >> (8 * (threadIdx.x & 3))) & 0xffu;
}

// Inclusive sums of v over the workgroup's threads, in thread order; the
// total in *total. `part` holds one double per wave.
__device__ __forceinline__ double block_scan(double v, double *part, double *total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_up(v, m, 64);
        if (lane >= m)
            v += o;
    }
    __syncthreads();
    if (lane == 63)
        part[wave] = v;
    __syncthreads();
    double before = 0.0, all = 0.0;
#pragma unroll
    for (int i = 0; i < kNT / 64; ++i) {
        if (i < wave)
            before += part[i];
        all += part[i];
    }
    *total = all;
    return before + v;
}

__device__ __forceinline__ int row_length(const VerifyParams &p, int b)
{
    if (p.idx && p.idx[b] < 0)
        return 0;
    return p.ctx ? clamp_len(p.ctx[b], p.num_tokens) : p.num_tokens;
}

__global__ __launch_bounds__(kNT) void ssu_verify_sums_kernel(const VerifyParams p, int chunks)
{
    __shared__ Walk w;
    __shared__ uint32_t bits[kNT / 4];
    __shared__ double part[kNT / 64];
    const int b = blockIdx.y, chunk = blockIdx.x;
    const int len = row_length(p, b);
    if (len == 0)
        return;
    if (threadIdx.x < 64)
        walk_row(p, b, len, w);
    __syncthreads();
    const int base = chunk * kVerifyChunk;
    const uint32_t gone = removed_bits(w, base, bits);
    double wt[kPer], sum = 0.0, total;
    weights8(p, b * p.t_bs + w.last * p.t_rs, b * p.d_bs + w.last * p.d_rs,
             base + threadIdx.x * kPer, w.subtract != 0, gone, wt);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        sum += wt[j];
    block_scan(sum, part, &total);
    if (threadIdx.x == 0)
        p.partial[(int64_t)b * (chunks + 1) + chunk] = total;
}

__global__ __launch_bounds__(kNT) void ssu_verify_draw_kernel(const VerifyParams p, int chunks)
{
    __shared__ Walk w;
    __shared__ uint32_t bits[kNT / 4];
    __shared__ double part[kNT / 64];
    __shared__ int pick;
    const int b = blockIdx.x, tid = threadIdx.x;
    const int len = row_length(p, b);
    if (len > 0) {
        if (tid < 64)
            walk_row(p, b, len, w);
        __syncthreads();
    }
    const int count = len > 0 ? w.count : 0;
    if (tid == 0)
        p.accepted[b] = count;
    if (p.path)
        for (int i = tid; i < p.max_accept; i += kNT)
            p.path[(int64_t)b * p.max_accept + i] = i < count ? w.path[i] : -1;
    if (len == 0) {
        if (tid == 0)
            p.next[b] = -1;
        return;
    }
    const double u = (double)p.uniforms[(int64_t)b * p.num_tokens];
    const int64_t t_off = b * p.t_bs + w.last * p.t_rs, d_off = b * p.d_bs + w.last * p.d_rs;
    double *sums = p.partial + (int64_t)b * (chunks + 1);

    // Attempt 0: the weights the first launch summed. Attempt 1, where they have
    // no mass: the target's row, summed here.
    for (int attempt = 0; attempt < 2; ++attempt) {
        const bool plain = attempt == 1;
        if (plain) {
            for (int c = 0; c < chunks; ++c) {
                double wt[kPer], sum = 0.0, all;
                weights8(p, t_off, d_off, c * kVerifyChunk + tid * kPer, false, 0, wt);
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    sum += wt[j];
                block_scan(sum, part, &all);
                if (tid == 0)
                    sums[c] = all;
            }
            __threadfence_block();
            __syncthreads();
        }
        // total, and the first chunk whose running sum passes u * total: chunks
        // in order, kNT at a time
        double total = 0.0;
        for (int c0 = 0; c0 < chunks; c0 += kNT) {
            double all;
            block_scan(c0 + tid < chunks ? sums[c0 + tid] : 0.0, part, &all);
            total += all;
        }
        if (!(total > 0.0))
            continue;
        const double goal = u * total;
        double before = 0.0, found_before = 0.0;
        int chunk = -1, last_chunk = 0;
        for (int c0 = 0; c0 < chunks && chunk < 0; c0 += kNT) {
            const double s = c0 + tid < chunks ? sums[c0 + tid] : 0.0;
            double all;
            const double incl = before + block_scan(s, part, &all);
            const uint64_t hit = __ballot(s > 0.0 && incl > goal);
            const uint64_t some = __ballot(s > 0.0);
            // first hit and last chunk with mass over the workgroup's waves
            __shared__ int hits[kNT / 64], somes[kNT / 64];
            __shared__ double pre;
            if ((tid & 63) == 0) {
                hits[tid >> 6] = hit ? c0 + tid + __ffsll((unsigned long long)hit) - 1 : -1;
                somes[tid >> 6] = some ? c0 + tid + 63 - __clzll((unsigned long long)some) : -1;
            }
            __syncthreads();
#pragma unroll
            for (int i = kNT / 64 - 1; i >= 0; --i)
                if (hits[i] >= 0)
                    chunk = hits[i];
#pragma unroll
            for (int i = 0; i < kNT / 64; ++i)
                if (somes[i] >= 0)
                    last_chunk = somes[i];
            if (chunk == c0 + tid)
                pre = incl - s;
            __syncthreads();
            if (chunk >= 0)
                found_before = pre;
            before += all;
            __syncthreads();
        }
        // nothing passes (u * total rounded up to the total): the last entry with mass
        const bool over = chunk < 0;
        if (over)
            chunk = last_chunk;
        const int base = chunk * kVerifyChunk;
        const uint32_t gone = plain ? 0u : removed_bits(w, base, bits);
        double wt[kPer], sum = 0.0, all;
        weights8(p, t_off, d_off, base + tid * kPer, !plain && w.subtract, gone, wt);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            sum += wt[j];
        const double incl = block_scan(sum, part, &all);
        // this thread's first entry past the goal, and its last with mass
        double run = found_before + (incl - sum);
        int first = -1, last = -1;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            run += wt[j];
            if (wt[j] > 0.0) {
                last = base + tid * kPer + j;
                if (first < 0 && !over && run > goal)
                    first = last;
            }
        }
        if (tid == 0)
            pick = -1;
        __syncthreads();
        if (last >= 0)
            atomicMax(&pick, last);
        __syncthreads();
        const int fallback = pick;
        __syncthreads();
        if (tid == 0)
            pick = 0x7fffffff;
        __syncthreads();
        if (first >= 0)
            atomicMin(&pick, first);
        __syncthreads();
        if (tid == 0)
            p.next[b] = pick == 0x7fffffff ? fallback : pick;
        return;
    }
    if (tid == 0)
        p.next[b] = -1;
}

}  // namespace

hipError_t launch_verify(const VerifyParams &p, hipStream_t stream)
{
    const int chunks = (p.vocab + kVerifyChunk - 1) / kVerifyChunk;
    (void)hipGetLastError();  // report only this launch's status
    hipLaunchKernelGGL(ssu_verify_sums_kernel, dim3((unsigned)chunks, (unsigned)p.batch), dim3(kNT),
                       0, stream, p, chunks);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(ssu_verify_draw_kernel, dim3((unsigned)p.batch), dim3(kNT), 0, stream, p,
                       chunks);
    return hipGetLastError();
}

}  // namespace ssu
