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

// Tokens from which chunks are taken. Token by token, time grows with the tokens; a chunk costs the
// same for 2 tokens as for all of its own. In a captured graph, us for 16 / 20 / 28 / 48 tokens one by one and in
// a chunk (bf16; the other types meet up to seven tokens later, by 5 us at most):
//   heads of 128: 32 of them 16.2 19.4 25.5 40.5 and 19.8; 512: 44 52 67 106 and 47; 2048: 133 164 223 370 and 147
//   heads of 256:  8 of them 23.3 28.2 38.6 58.2 and 17.4; 128: 40 47 59 91 and 31; 512: 130 153 199 316 and 102
//   heads of 64:   8 of them 16.6 20.0 26.1 41.4 and 16.4; 128: 16.0 19.1 25.1 39.7 and 18.9; 512: 17.4 20.5 26.3 41.6 and 32.5
//   heads of 32:   8 of them 11.0 13.0 16.7 25.7 and 14.8; 128: 11.3 13.3 17.3 26.4 and 16.8; 512: 11.7 13.7 17.9 27.7 and 29.0
int least_tokens(int64_t heads, int64_t d)
{
    if (d >= 128)
        return 18;
    return d == 64 ? (heads > 256 ? 36 : 18) : (heads > 256 ? 50 : 24);
}
// Bytes handed over at a time: 8 x 4096 tokens of 32 heads of 128 take 724 us by 96 MiB, 683 by 256, 662
// by 512; 8 x 777 of fp16 182, 173 and 172: each segment fills and drains the GPU twice.
constexpr int64_t kDeltaSegment = (int64_t)256 << 20;

}  // namespace

DeltaPlan delta_plan(int64_t batch, int64_t hq, int64_t hv, int64_t d, int64_t seq_len, int32_t io_dtype)
{
    DeltaPlan q = {};
    if (batch <= 0 || batch > 65535 || seq_len < least_tokens(batch * hv, d))
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
    // beyond, those of 128 fetch a chunk for eight waves. 2048 tokens of 32 heads of 128, bf16: 205 against 251
    // us at 256 of the former, 342 against 261 at 320, 410 against 343 at 512; 1024 of fp16 132 against 169 at 256,
    // 262 against 213 at 512; 512 of fp32 85 against 107 and 169 against 143.
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
    if (q.spans && p.workspace && delta_rows_aligned(p, 16)) {
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
