// Depthwise causal convolution over a paged pool of conv states:
//   out[b,t,c] = act(bias[c] + sum_j weight[c,j] win[t+j]),
// win = the W-1 inputs kept in the pool followed by x, then the pool's row is
// left with the last W-1 inputs of the row's L_b tokens.
//
// Mapping: a thread owns one channel and kTile consecutive tokens and keeps
// the last W inputs in registers, so every input is loaded once per tile (plus
// W-1 inputs in front of it). The first tile of a row is the only one that
// reads the pool and the only one that writes it, after its reads, so no other
// thread of the launch sees a row half updated.
#include "ssu_device.h"
#include "ssu_internal.h"

namespace ssu {
namespace {

constexpr int kMaxW = 8;
constexpr int kTile = 16;

__global__ __launch_bounds__(256) void ssu_conv_kernel(const ConvParams p)
{
    const int c = blockIdx.x * 256 + threadIdx.x;
    const int t0 = blockIdx.y * kTile;
    const int b = blockIdx.z;
    if (c >= p.channels)
        return;
    const int t1 = min(t0 + kTile, p.seq_len);
    const int64_t xo = (int64_t)b * p.x_bs + c;
    const int64_t oo = (int64_t)b * p.out_bs + c;
    const int row = p.idx ? p.idx[b] : b;
    const int len = row < 0 ? 0 : (p.ctx ? clamp_len(p.ctx[b], p.seq_len) : p.seq_len);
    const int taps = p.width - 1;
    const int64_t so = (int64_t)row * p.st_row + (int64_t)c * p.st_chan;

    // the window's input i (0: the oldest in the pool; taps: the first of x)
    auto input = [&](int i) {
        return i < taps ? ld_io(p.state, so + i * p.st_tap, p.state_dtype)
                        : ld_io(p.x, xo + (int64_t)(i - taps) * p.x_ts, p.io_dtype);
    };
    // the row's new state, read before anything is written (out may be x)
    const bool keeps = p.update && t0 == 0 && len > 0;
    float keep[kMaxW] = {};
    if (keeps) {
#pragma unroll
        for (int j = 0; j < kMaxW; ++j)
            keep[j] = j < taps ? input(len + j) : 0.0f;
    }
    if (p.out) {
        float w[kMaxW], win[kMaxW];
#pragma unroll
        for (int j = 0; j < kMaxW; ++j) {
            w[j] = j < p.width ? ld_io(p.weight, (int64_t)c * p.width + j, p.weight_dtype) : 0.0f;
            win[j] = j < taps && t0 < len ? input(t0 + j) : 0.0f;
        }
        const float bias = p.bias ? ld_io(p.bias, c, p.weight_dtype) : 0.0f;
        for (int t = t0; t < t1; ++t) {
            float y = 0.0f;
            if (t < len) {
                const float in = ld_io(p.x, xo + (int64_t)t * p.x_ts, p.io_dtype);
                y = bias;
#pragma unroll
                for (int j = 0; j < kMaxW; ++j) {
                    if (j == taps)
                        win[j] = in;
                    y = fmaf(w[j], win[j], y);
                }
#pragma unroll
                for (int j = 0; j + 1 < kMaxW; ++j)
                    win[j] = win[j + 1];
                if (p.silu)
                    y = silu_f32(y);
            }
            st_io(p.out, oo + (int64_t)t * p.out_ts, y, p.io_dtype);
        }
    }
    if (keeps) {
#pragma unroll
        for (int j = 0; j < kMaxW; ++j)
            if (j < taps)
                st_io(p.state, so + j * p.st_tap, keep[j], p.state_dtype);
    }
}

}  // namespace

hipError_t launch_conv(const ConvParams &p, hipStream_t stream)
{
    const unsigned tiles = p.out ? (unsigned)((p.seq_len + kTile - 1) / kTile) : 1u;
    if (p.batch > 65535 || tiles > 65535)
        return hipErrorInvalidConfiguration;
    (void)hipGetLastError();  // report only this launch's status
    hipLaunchKernelGGL(ssu_conv_kernel, dim3((unsigned)((p.channels + 255) / 256), tiles, p.batch),
                       dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace ssu
