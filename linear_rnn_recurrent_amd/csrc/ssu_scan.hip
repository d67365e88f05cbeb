// Per-channel selective scan over a paged state pool, for prompts and single
// tokens:
//   dt' = dt + dt_bias (softplus);  h[d,n] = h[d,n] exp(A[d,n] dt') + B[n] dt' x[d]
//   out[d] = (sum_n h[d,n] C[n] + D[d] x[d]) silu(z[d])
//
// Three evaluations, by the sizes (scan_plan in ssu_scan_plan.h):
//
// Rows (ssu_scan_rows.hip; single tokens, windows, many rows of a few tokens):
// LPC lanes share a channel, four state entries each, so that the state, of a
// single token all but a few percent of the bytes, is read and written in whole
// cache lines; the sum over dstate is a butterfly across the channel's lanes.
// Single tokens are bound by HBM.
//
// Sweep (ssu_scan_prompt.h; prompts with channels enough to fill the GPU): a
// workgroup takes 16 channels through the tokens, its waves side by side along
// them. Every wave runs its 8 or 16 tokens of a step from a zero start, keeping the
// decays in registers; the ends meet in LDS; then the tokens run again from
// their true start. Per token, channel and state entry that is a product, an
// exponential at half rate, two products with B and two multiply-adds for the
// state, one for the output: 8 issue slots of the vector ALU, which bounds it (11
// counted, with softplus, gate and exchange: busy 72% of 57 us at 8 x 777 x 2560 with
// the uneven lengths that the counters were taken with; 50 to 74 us by the lengths).
//
// Chunks (ssu_scan_prompt.h; long prompts of few channels): a lane is a channel
// and holds 16 state entries, which makes B and C the same for the whole wave
// (scalar registers, no lane traffic) and the sum over dstate private to the
// lane: 6 slots. The tokens are cut into chunks that run side by side:
//   pack    B and C of every token in fp32, padded to 16 states (scalar loads)
//   ends    every chunk's state from a zero start, and its sum of dt'
//           (the chunk's decay is exp(A sum dt'))
//   tokens  every chunk's start from the pool's state and the ends before it, in
//           order, then its tokens: the outputs, the last state
// The chunks' decays are computed twice (11 slots; 1 x 2048 x 5120: pack 5 us, ends
// 42 of which the vector ALU 29, tokens 64 of which 42). dstate above 16 takes
// ceil(dstate / 16) waves, whose partial outputs meet in LDS. (A single chunk
// needs no ends; without outputs a small kernel folds the ends into the last
// state and the tokens are not run.)
#include "ssu_scan_impl.h"

namespace ssu {

hipError_t launch_scan_rows(const ScanParams &p, hipStream_t stream);
hipError_t launch_scan_prompt_f32(const ScanParams &p, const ScanPlan &q, hipStream_t stream);
hipError_t launch_scan_prompt_f16(const ScanParams &p, const ScanPlan &q, hipStream_t stream);
hipError_t launch_scan_prompt_bf16(const ScanParams &p, const ScanPlan &q, hipStream_t stream);

int64_t scan_workspace_floats(int64_t batch, int64_t dim, int64_t dstate, int64_t ngroups,
                              int64_t seq_len)
{
    if (batch <= 0 || seq_len <= 0)
        return 0;  // nothing runs
    int64_t most = 0;  // with and without context_lengths
    for (int ragged = 0; ragged < 2; ++ragged) {
        const ScanPlan q = scan_plan(batch, dim, dstate, ngroups, seq_len, ragged != 0);
        const int64_t floats = q.bc_floats + q.start_floats + q.sum_floats;
        most = floats > most ? floats : most;
    }
    return most;
}

hipError_t launch_scan(const ScanParams &p, hipStream_t stream)
{
    (void)hipGetLastError();  // report only this launch's status
    ScanPlan q = scan_plan(p.batch, p.dim, p.dstate, p.ngroups, p.seq_len, p.ctx != nullptr);
    if (!q.rows) {
        q.s.bc = p.workspace;
        q.s.zeros = q.bc_floats - 2 * kStates;
        q.s.start = q.s.bc + q.bc_floats;
        q.s.sum = q.s.start + q.start_floats;
        switch (p.io_dtype) {
        case kF32: return launch_scan_prompt_f32(p, q, stream);
        case kF16: return launch_scan_prompt_f16(p, q, stream);
        default: return launch_scan_prompt_bf16(p, q, stream);
        }
    }
    return launch_scan_rows(p, stream);
}

}  // namespace ssu
