// The gated delta rule on given q, k and v over a paged state pool:
//   S <- alpha S;  u = beta (v - S k);  S <- S + u k^T;  o = scale S q
//
// Two evaluations, by the sizes (delta_plan): token by token (ssu_delta_rows.h; single
// tokens, windows, unaligned rows) and in chunks of 64 or 32 tokens on the matrix cores
// (ssu_delta_chunks.h; prompts).
#include "ssu_delta_impl.h"

namespace ssu {

hipError_t launch_delta_rows_f32(const DeltaParams &p, hipStream_t stream);
hipError_t launch_delta_rows_f16(const DeltaParams &p, hipStream_t stream);
hipError_t launch_delta_rows_bf16(const DeltaParams &p, hipStream_t stream);
hipError_t launch_delta_chunks_f32(const DeltaParams &p, const DeltaPlan &plan, hipStream_t stream);
hipError_t launch_delta_chunks_f16(const DeltaParams &p, const DeltaPlan &plan, hipStream_t stream);
hipError_t launch_delta_chunks_bf16(const DeltaParams &p, const DeltaPlan &plan, hipStream_t stream);

namespace {

// Tokens from which chunks are taken: a single chunk takes 19 us of one row of 32 heads of
// 128, 43 of 16 rows, 135 of 64; token by token 16 of them take 16, 44 and 134 us, 31 take 28, 72
// and 250.
constexpr int kDeltaLeast = 18;
// Bytes handed over at a time: 8 x 4096 tokens of 32 heads take 814 us by 48 MiB, 672 by
// 96, 601 by 192, 583 by 400, 564 at once (3.4 GB): each segment fills and drains the GPU twice.
constexpr int64_t kDeltaSegment = (int64_t)256 << 20;

}  // namespace

DeltaPlan delta_plan(int64_t batch, int64_t hq, int64_t hv, int64_t d, int64_t seq_len, int32_t io_dtype)
{
    DeltaPlan q = {};
    if (batch <= 0 || batch > 65535 || seq_len < kDeltaLeast)
        return q;
    const int planes = delta_planes(io_dtype), tiles = delta_tiles(d, planes);
    q.spans = (int32_t)((seq_len + 63) / 64);
    const int64_t kq = batch * hq * 256 * d * planes;
    const int64_t head = batch * hv * (4 / tiles) * delta_head_bytes(tiles);
    int64_t segment = kDeltaSegment / (kq + head);
    segment = segment < 1 ? 1 : segment;
    const int64_t parts = (q.spans + segment - 1) / segment;
    segment = (q.spans + parts - 1) / parts;  // of like sizes
    q.segment = (int32_t)segment;
    // Workgroups of 64 value columns, as long as each has a CU to itself, run a chunk faster;
    // beyond, those of 128 fetch a chunk for eight waves: 169 against 206 us at 256 of the former (4
    // x 2048 tokens, 32 heads of 128), 283 against 221 at 320, 347 against 297 at 512.
    q.wide = batch * hv * d > 256 * 64;
    q.kq_bytes = kq * segment;
    q.head_bytes = head * segment;
    q.carry_bytes = segment < q.spans ? 4 * batch * hv * d * d : 0;
    return q;
}

int64_t delta_workspace_bytes(int64_t batch, int64_t hq, int64_t hv, int64_t d, int64_t seq_len,
                              int32_t io_dtype)
{
    const DeltaPlan q = delta_plan(batch, hq, hv, d, seq_len, io_dtype);
    return q.spans ? q.kq_bytes + q.head_bytes + q.carry_bytes : 0;
}

hipError_t launch_delta(const DeltaParams &p, hipStream_t stream)
{
    (void)hipGetLastError();  // report only this launch's status
    const DeltaPlan q = delta_plan(p.batch, p.hq, p.hv, p.d, p.seq_len, p.io_dtype);
    if (q.spans && p.workspace && delta_rows_aligned(p, 16, true)) {
        switch (p.io_dtype) {
        case kF32: return launch_delta_chunks_f32(p, q, stream);
        case kF16: return launch_delta_chunks_f16(p, q, stream);
        default: return launch_delta_chunks_bf16(p, q, stream);
        }
    }
    switch (p.io_dtype) {
    case kF32: return launch_delta_rows_f32(p, stream);
    case kF16: return launch_delta_rows_f16(p, stream);
    default: return launch_delta_rows_bf16(p, stream);
    }
}

}  // namespace ssu
