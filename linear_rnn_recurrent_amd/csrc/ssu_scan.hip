// Per-channel selective scan over a paged state pool, for prompts and single
// tokens:
//   dt' = dt + dt_bias (softplus);  h[d,n] = h[d,n] exp(A[d,n] dt') + B[n] dt' x[d]
//   out[d] = (sum_n h[d,n] C[n] + D[d] x[d]) silu(z[d])
//
// Mapping: LPC lanes share a channel, four state entries each (lanes past
// dstate idle with zeros), and keep them in registers over all tokens; the sum
// over dstate is a butterfly across the channel's lanes.
#include "ssu_device.h"
#include "ssu_internal.h"

namespace ssu {
namespace {

template <int LPC>
__global__ __launch_bounds__(256) void ssu_scan_kernel(const ScanParams p)
{
    constexpr int CH = 256 / LPC;  // channels per workgroup
    const int sub = threadIdx.x & (LPC - 1);
    const int ch = threadIdx.x / LPC;
    const int tiles = (p.dim + CH - 1) / CH;
    const int b = blockIdx.x / tiles;
    const int d_raw = (blockIdx.x - b * tiles) * CH + ch;
    const int d = min(d_raw, p.dim - 1);
    const int n0 = sub * 4;
    const bool own = n0 < p.dstate;
    const bool writes = own && d_raw < p.dim;
    const bool head = sub == 0 && d_raw < p.dim;
    const int row = p.idx ? p.idx[b] : b;
    const int len = row < 0 ? 0 : (p.ctx ? clamp_len(p.ctx[b], p.seq_len) : p.seq_len);
    const int g = d / (p.dim / p.ngroups);
    const int64_t so = (int64_t)row * p.row_stride + (int64_t)d * p.dstate + n0;

    float h[4] = {}, a[4] = {};
    if (own && len > 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = p.A[(int64_t)d * p.dstate + n0 + j];
            h[j] = ld_io(p.state, so + j, p.state_dtype);
        }
    }
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.0f;
    const float skip = p.D ? p.D[d] : 0.0f;
    for (int t = 0; t < len; ++t) {
        float v = ld_io(p.dt, b * p.dt_bs + t * p.dt_ts + d, p.dt_dtype) + bias;
        if (p.dt_softplus)
            v = softplus_f32(v);
        const float x = ld_io(p.x, b * p.x_bs + t * p.x_ts + d, p.io_dtype);
        const int64_t bo = b * p.b_bs + t * p.b_ts + (int64_t)g * p.dstate + n0;
        const int64_t co = b * p.c_bs + t * p.c_ts + (int64_t)g * p.dstate + n0;
        const float u = v * x;
        float y = 0.0f;
        if (own) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = fmaf(u, ld_io(p.B, bo + j, p.bc_dtype), h[j] * expf(a[j] * v));
                if (p.out)
                    y = fmaf(h[j], ld_io(p.C, co + j, p.bc_dtype), y);
            }
        }
        if (p.out) {
            y = group_sum<LPC>(y);
            if (head) {
                y = fmaf(skip, x, y);
                if (p.z)
                    y *= silu_f32(ld_io(p.z, b * p.z_bs + t * p.z_ts + d, p.io_dtype));
                st_io(p.out, b * p.out_bs + t * p.out_ts + d, y, p.io_dtype);
            }
        }
    }
    if (p.out && head)
        for (int t = len; t < p.seq_len; ++t)
            st_io(p.out, b * p.out_bs + t * p.out_ts + d, 0.0f, p.io_dtype);
    if (p.update && writes && len > 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            st_io(p.state, so + j, h[j], p.state_dtype);
    }
}

template <int LPC>
hipError_t launch_scan_lanes(const ScanParams &p, hipStream_t stream)
{
    const int64_t blocks = (int64_t)p.batch * ((p.dim + 256 / LPC - 1) / (256 / LPC));
    if (blocks > 0x7fffffff)
        return hipErrorInvalidConfiguration;
    (void)hipGetLastError();  // report only this launch's status
    hipLaunchKernelGGL(ssu_scan_kernel<LPC>, dim3((unsigned)blocks), dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_scan(const ScanParams &p, hipStream_t stream)
{
    if (p.dstate <= 4) return launch_scan_lanes<1>(p, stream);
    if (p.dstate <= 8) return launch_scan_lanes<2>(p, stream);
    if (p.dstate <= 16) return launch_scan_lanes<4>(p, stream);
    if (p.dstate <= 32) return launch_scan_lanes<8>(p, stream);
    if (p.dstate <= 64) return launch_scan_lanes<16>(p, stream);
    if (p.dstate <= 128) return launch_scan_lanes<32>(p, stream);
    return launch_scan_lanes<64>(p, stream);
}

}  // namespace ssu
