// Depthwise causal convolution over a paged pool of conv states:
//   out[b,t,c] = act(bias[c] + sum_j weight[c,j] win[t+j]),
// win = the W-1 inputs kept in the pool followed by x, then the pool's row is
// left with the last W-1 inputs of the row's L_b tokens.
//
// Mapping: a thread owns V adjacent channels (16 bytes of x where alignment
// allows) and a tile of consecutive tokens, and slides the window through
// registers: every input is loaded once per tile, plus the W-1 inputs in front
// of it. Loads run a batch of kU tokens ahead of their use. The op reads and
// writes each activation once and is bound by HBM; the weights and the pool are
// read in whole vectors too (one element at a time they cost more than the
// tokens: 31 us instead of 21 at 8 x 512 x 5376). The first tile of a row is the
// only one that reads the pool and the only one that writes it, after its reads,
// so no other thread of the launch sees a row half updated.
// Measured, bf16, W 4 (8 x 512 x 5376 with uneven lengths | 1 x 4099 x 5120):
// 16.5 | 19.5 us, 4.2 | 4.3 TB/s; tiles of 16 tokens 20.5 | 19.3; one or four
// tokens loaded together 17.3 | 21.8 and 17.2 | 20.2; cached stores 17.2 | 21.8;
// neighbouring tiles kept on one XCD 20.0 | 22.4 (uneven rows meet on an XCD).
#include "ssu_device.h"
#include "ssu_internal.h"

namespace ssu {
namespace {

constexpr int kMaxW = 8;
constexpr int kU = 2;     // tokens loaded together
constexpr int kTile = 8;  // tokens of a thread: at least the W - 1 in front of it

// V adjacent elements of storage type T: raw bits, and their values.
template <typename T, int V>
struct Pack {
    static constexpr int BYTES = V * (sizeof(T) == 4 ? 4 : 2);
    static constexpr int WORDS = BYTES >= 4 ? BYTES / 4 : 1;
    uint32_t w[WORDS];

    __device__ __forceinline__ void load(const void *p, int64_t i)
    {
        const char *q = static_cast<const char *>(p) + i * (BYTES / V);
        if constexpr (BYTES == 2) {
            w[0] = *reinterpret_cast<const uint16_t *>(q);
        } else if constexpr (BYTES == 16) {
            const u32x4 v = *reinterpret_cast<const u32x4 *>(q);
            w[0] = v[0], w[1] = v[1], w[2] = v[2], w[3] = v[3];
        } else if constexpr (BYTES == 8) {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(q);
            w[0] = v[0], w[1] = v[1];
        } else {
            w[0] = *reinterpret_cast<const uint32_t *>(q);
        }
    }
    __device__ __forceinline__ float get(int k) const
    {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[k]);
        else
            return cvt_raw1<T>(k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xffffu);
    }
    __device__ __forceinline__ void set(const float (&v)[V])
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int k = 0; k < V; ++k)
                w[k] = __float_as_uint(v[k]);
        } else {
            uint16_t e[V];
#pragma unroll
            for (int k = 0; k < V; ++k)
                e[k] = __is_same(T, bf16_t) ? __builtin_bit_cast(uint16_t, (__bf16)v[k])
                                            : __builtin_bit_cast(uint16_t, (_Float16)v[k]);
#pragma unroll
            for (int k = 0; k < WORDS; ++k)
                w[k] = e[2 * k] | (2 * k + 1 < V ? (uint32_t)e[(2 * k + 1) % V] << 16 : 0u);
        }
    }
    // past the caches, for outputs (16 bytes; smaller ones as they are)
    __device__ __forceinline__ void stream(void *p, int64_t i) const
    {
        if constexpr (BYTES == 16)
            __builtin_nontemporal_store(
                u32x4{w[0], w[1], w[2], w[3]},
                reinterpret_cast<u32x4 *>(static_cast<char *>(p) + i * (BYTES / V)));
        else
            store(p, i);
    }
    __device__ __forceinline__ void store(void *p, int64_t i) const
    {
        char *q = static_cast<char *>(p) + i * (BYTES / V);
        if constexpr (BYTES == 2)
            *reinterpret_cast<uint16_t *>(q) = (uint16_t)w[0];
        else if constexpr (BYTES == 16)
            *reinterpret_cast<u32x4 *>(q) = u32x4{w[0], w[1], w[2], w[3]};
        else if constexpr (BYTES == 8)
            *reinterpret_cast<u32x2 *>(q) = u32x2{w[0], w[1]};
        else
            *reinterpret_cast<uint32_t *>(q) = w[0];
    }
};

// v sigmoid(v) on the hardware exp2 and reciprocal (1 ulp each).
__device__ __forceinline__ float silu_hw(float v)
{
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * 1.4426950408889634f));
}

// N adjacent elements of storage type T at element offset i as floats: in
// 16-byte (8-byte) pieces where `vec` says that i and the base allow it.
template <typename T, int N>
__device__ __forceinline__ void ld_run(const void *p, int64_t i, bool vec, float (&v)[N])
{
    constexpr int ES = sizeof(T) == 4 ? 4 : 2, PER = N * ES % 16 == 0 ? 16 / ES : 8 / ES;
    if constexpr (N % PER == 0) {
        if (vec) {
            Pack<T, PER> w[N / PER];
#pragma unroll
            for (int k = 0; k < N / PER; ++k)
                w[k].load(p, i + k * PER);
#pragma unroll
            for (int k = 0; k < N; ++k)
                v[k] = w[k / PER].get(k % PER);
            return;
        }
    }
    Pack<T, 1> w[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
        w[k].load(p, i + k);
#pragma unroll
    for (int k = 0; k < N; ++k)
        v[k] = w[k].get(0);
}
template <typename T, int N>
__device__ __forceinline__ void st_run(void *p, int64_t i, bool vec, const float (&v)[N])
{
    constexpr int ES = sizeof(T) == 4 ? 4 : 2, PER = N * ES % 16 == 0 ? 16 / ES : 8 / ES;
    if constexpr (N % PER == 0) {
        if (vec) {
#pragma unroll
            for (int k = 0; k < N / PER; ++k) {
                float e[PER];
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    e[j] = v[k * PER + j];
                Pack<T, PER> w;
                w.set(e);
                w.store(p, i + k * PER);
            }
            return;
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float e[1] = {v[k]};
        Pack<T, 1> w;
        w.set(e);
        w.store(p, i + k);
    }
}
// The same for a type that is a (uniform) argument.
template <int N>
__device__ __forceinline__ void ld_run_dt(const void *p, int64_t i, int dt, bool vec, float (&v)[N])
{
    if (dt == kF32)
        ld_run<float, N>(p, i, vec, v);
    else if (dt == kBF16)
        ld_run<bf16_t, N>(p, i, vec, v);
    else
        ld_run<_Float16, N>(p, i, vec, v);
}
template <int N>
__device__ __forceinline__ void st_run_dt(void *p, int64_t i, int dt, bool vec, const float (&v)[N])
{
    if (dt == kF32)
        st_run<float, N>(p, i, vec, v);
    else if (dt == kBF16)
        st_run<bf16_t, N>(p, i, vec, v);
    else
        st_run<_Float16, N>(p, i, vec, v);
}

struct ConvShape {
    int32_t cols, tiles;  // column groups of V channels; tiles a row
    uint32_t row_blocks;  // workgroups a row
    // the pool's layout: the W-1 taps of a channel adjacent and channels dense,
    // the channels of a tap adjacent, or neither; runs of V aligned for vectors
    int32_t layout;
    bool w_vec, s_vec;
};
enum : int { kAny = 0, kTapsInside = 1, kChannelsInside = 2 };

// The pool's V channels, [tap][channel].
template <int V, int TAPS>
__device__ __forceinline__ void ld_taps(const ConvParams &p, const ConvShape &s, int64_t so,
                                        float (&old)[TAPS][V])
{
    if (s.layout == kTapsInside) {
        float run[V * TAPS];
        ld_run_dt<V * TAPS>(p.state, so, p.state_dtype, s.s_vec, run);
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int j = 0; j < TAPS; ++j)
                old[j][k] = run[k * TAPS + j];
    } else if (s.layout == kChannelsInside) {
#pragma unroll
        for (int j = 0; j < TAPS; ++j)
            ld_run_dt<V>(p.state, so + j * p.st_tap, p.state_dtype, s.s_vec, old[j]);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int j = 0; j < TAPS; ++j)
                old[j][k] = ld_io(p.state, so + k * p.st_chan + j * p.st_tap, p.state_dtype);
    }
}
template <int V, int TAPS>
__device__ __forceinline__ void st_taps(const ConvParams &p, const ConvShape &s, int64_t so,
                                        const float (&now)[TAPS][V])
{
    if (s.layout == kTapsInside) {
        float run[V * TAPS];
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int j = 0; j < TAPS; ++j)
                run[k * TAPS + j] = now[j][k];
        st_run_dt<V * TAPS>(p.state, so, p.state_dtype, s.s_vec, run);
    } else if (s.layout == kChannelsInside) {
#pragma unroll
        for (int j = 0; j < TAPS; ++j)
            st_run_dt<V>(p.state, so + j * p.st_tap, p.state_dtype, s.s_vec, now[j]);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int j = 0; j < TAPS; ++j)
                st_io(p.state, so + k * p.st_chan + j * p.st_tap, now[j][k], p.state_dtype);
    }
}

// W: the width.
template <typename T, int V, int W>
__global__ __launch_bounds__(256) void ssu_conv_kernel(const ConvParams p, const ConvShape s)
{
    const int b = blockIdx.x / s.row_blocks;
    const int64_t i = (int64_t)(blockIdx.x - b * s.row_blocks) * 256 + threadIdx.x;
    if (i >= (int64_t)s.cols * s.tiles)
        return;
    const int col = (int)(i % s.cols), c = col * V;
    const int t0 = (int)(i / s.cols) * kTile, t1 = min(t0 + kTile, p.seq_len);
    const int64_t xo = b * p.x_bs + c, oo = b * p.out_bs + c;
    const int row = p.idx ? p.idx[b] : b;
    const int len = row < 0 ? 0 : (p.ctx ? clamp_len(p.ctx[b], p.seq_len) : p.seq_len);
    constexpr int TAPS = W - 1;
    const int64_t so = (int64_t)row * p.st_row + (int64_t)c * p.st_chan;
    const int end = min(t1, len);

    constexpr int NT = TAPS > 0 ? TAPS : 1;
    Pack<T, V> next[kU];
    if (t0 < end && p.out) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
            next[u].load(p.x, xo + (int64_t)min(t0 + u, end - 1) * p.x_ts);
    }
    // the pool's inputs, and the row's new ones, read before anything is
    // written (out may be x)
    const bool keeps = TAPS > 0 && p.update && t0 == 0 && len > 0;
    float old[NT][V], keep[NT][V];
    if constexpr (TAPS > 0) {
        if (t0 == 0 && len > 0)
            ld_taps<V, TAPS>(p, s, so, old);
        if (keeps) {
            Pack<T, V> in[TAPS];
#pragma unroll
            for (int j = 0; j < TAPS; ++j)
                in[j].load(p.x, xo + (int64_t)max(len + j - TAPS, 0) * p.x_ts);
#pragma unroll
            for (int j = 0; j < TAPS; ++j)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    keep[j][k] = in[j].get(k);
                    // fewer tokens than taps: old inputs move up
#pragma unroll
                    for (int o = j + 1; o < TAPS; ++o)
                        keep[j][k] = len + j == o ? old[o][k] : keep[j][k];
                }
        }
    }
    if (p.out) {
        float win[W][V], w[W][V], bias[V];
        if (t0 < end) {
            float run[V * W];
            ld_run_dt<V * W>(p.weight, (int64_t)c * W, p.weight_dtype, s.w_vec, run);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                bias[k] = 0.0f;
#pragma unroll
                for (int j = 0; j < W; ++j)
                    w[j][k] = run[k * W + j];
            }
            if (p.bias)
                ld_run_dt<V>(p.bias, c, p.weight_dtype, s.w_vec, bias);
            if constexpr (TAPS > 0) {
                Pack<T, V> in[TAPS];  // tiles are longer than the window: all of x, or all the pool's
                if (t0 > 0) {
#pragma unroll
                    for (int j = 0; j < TAPS; ++j)
                        in[j].load(p.x, xo + (int64_t)(t0 + j - TAPS) * p.x_ts);
                }
#pragma unroll
                for (int j = 0; j < TAPS; ++j)
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        win[j][k] = t0 > 0 ? in[j].get(k) : old[j][k];
            }
        }
        for (int t = t0; t < end; t += kU) {
            Pack<T, V> now[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u)
                now[u] = next[u];
            if (t + kU < end) {
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    next[u].load(p.x, xo + (int64_t)min(t + kU + u, end - 1) * p.x_ts);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (t + u >= end)
                    break;
                float y[V];
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    win[TAPS][k] = now[u].get(k);
                    float acc = bias[k];
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        acc = fmaf(w[j][k], win[j][k], acc);
#pragma unroll
                    for (int j = 0; j < TAPS; ++j)
                        win[j][k] = win[j + 1][k];
                    y[k] = p.silu ? silu_hw(acc) : acc;
                }
                Pack<T, V> o;
                o.set(y);
                o.stream(p.out, oo + (int64_t)(t + u) * p.out_ts);
            }
        }
        Pack<T, V> zero;
#pragma unroll
        for (int k = 0; k < Pack<T, V>::WORDS; ++k)
            zero.w[k] = 0;
        for (int t = max(t0, len); t < t1; ++t)
            zero.stream(p.out, oo + (int64_t)t * p.out_ts);
    }
    if constexpr (TAPS > 0) {
        if (keeps)
            st_taps<V, TAPS>(p, s, so, keep);
    }
}

template <typename T, int V, int W>
hipError_t launch_conv_cfg(const ConvParams &p, hipStream_t stream)
{
    static_assert(kTile >= kMaxW - 1, "the inputs in front of a tile lie in the one before it");
    ConvShape s;
    s.cols = p.channels / V;
    s.tiles = p.out ? (p.seq_len + kTile - 1) / kTile : 1;
    const int wes = p.weight_dtype == kF32 ? 4 : 2, ses = p.state_dtype == kF32 ? 4 : 2;
    auto run_bytes = [](int bytes) { return bytes % 16 == 0 ? 16 : 8; };  // a piece of a run
    s.w_vec = (V * wes) % 8 == 0 && (uintptr_t)p.weight % 16 == 0 && (uintptr_t)p.bias % 16 == 0;
    s.layout = p.st_tap == 1 && p.st_chan == W - 1 ? kTapsInside
               : p.st_chan == 1                   ? kChannelsInside
                                                  : kAny;
    const int piece = run_bytes(V * ses * (s.layout == kTapsInside ? W - 1 : 1));
    s.s_vec = (V * ses) % 8 == 0 && (uintptr_t)p.state % piece == 0 && p.st_row * ses % piece == 0 &&
              (s.layout == kTapsInside || p.st_tap * ses % piece == 0);
    const int64_t blocks = ((int64_t)s.cols * s.tiles + 255) / 256;
    if (!launchable((__int128)blocks * p.batch, 256))
        return hipErrorInvalidConfiguration;
    s.row_blocks = (uint32_t)blocks;
    hipLaunchKernelGGL((ssu_conv_kernel<T, V, W>), dim3((unsigned)(blocks * p.batch)), dim3(256), 0, stream, p, s);
    return hipGetLastError();
}

template <typename T, int V>
hipError_t launch_conv_width(const ConvParams &p, hipStream_t stream)
{
    switch (p.width) {
    case 1: return launch_conv_cfg<T, V, 1>(p, stream);
    case 2: return launch_conv_cfg<T, V, 2>(p, stream);
    case 3: return launch_conv_cfg<T, V, 3>(p, stream);
    case 4: return launch_conv_cfg<T, V, 4>(p, stream);
    case 5: return launch_conv_cfg<T, V, 5>(p, stream);
    case 6: return launch_conv_cfg<T, V, 6>(p, stream);
    case 7: return launch_conv_cfg<T, V, 7>(p, stream);
    default: return launch_conv_cfg<T, V, 8>(p, stream);
    }
}

// As many channels a thread as x's and out's alignment allows.
template <typename T>
hipError_t launch_conv_type(const ConvParams &p, hipStream_t stream)
{
    constexpr int ES = sizeof(T) == 4 ? 4 : 2, MOST = 16 / ES;
    auto fits = [&](int v) {
        return p.channels % v == 0 && (uintptr_t)p.x % (v * ES) == 0 &&
               (uintptr_t)p.out % (v * ES) == 0 && p.x_bs % v == 0 && p.x_ts % v == 0 &&
               p.out_bs % v == 0 && p.out_ts % v == 0;
    };
    if (fits(MOST))
        return launch_conv_width<T, MOST>(p, stream);
    if (fits(2))
        return launch_conv_width<T, 2>(p, stream);
    return launch_conv_width<T, 1>(p, stream);
}

}  // namespace

hipError_t launch_conv(const ConvParams &p, hipStream_t stream)
{
    (void)hipGetLastError();  // report only this launch's status
    switch (p.io_dtype) {
    case kF32: return launch_conv_type<float>(p, stream);
    case kF16: return launch_conv_type<_Float16>(p, stream);
    default: return launch_conv_type<bf16_t>(p, stream);
    }
}

}  // namespace ssu
