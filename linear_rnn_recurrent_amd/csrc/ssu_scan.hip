// Per-channel selective scan over a paged state pool, for prompts and single
// tokens:
//   dt' = dt + dt_bias (softplus);  h[d,n] = h[d,n] exp(A[d,n] dt') + B[n] dt' x[d]
//   out[d] = (sum_n h[d,n] C[n] + D[d] x[d]) silu(z[d])
//
// Three evaluations, by the sizes (scan_plan):
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
// counted, with softplus, gate and exchange: busy 72% of 57 us at 8 x 777 x 2560).
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
#include <math.h>

#include "ssu_scan_impl.h"

namespace ssu {

hipError_t launch_scan_rows(const ScanParams &p, hipStream_t stream);
hipError_t launch_scan_prompt_f32(const ScanParams &p, const ScanPlan &q, hipStream_t stream);
hipError_t launch_scan_prompt_f16(const ScanParams &p, const ScanPlan &q, hipStream_t stream);
hipError_t launch_scan_prompt_bf16(const ScanParams &p, const ScanPlan &q, hipStream_t stream);

namespace {

// Estimated microseconds of the three evaluations, fitted to measurements of each
// at 37 sizes (bf16, 1 to 64 rows, 17 to 8192 tokens, 160 to 8192 channels, dstate
// 16 to 256: nearly all within 25%; where B and C are not aligned to four entries
// rows take twice as long and sweeps a quarter longer). `mega` counts 1e6 state
// entries and tokens, `tiles` the sixteens of dstate. Rows of uneven lengths, an
// eighth of seq_len up, take a share of it: the sweep's, longest first and in short
// steps, least; of the chunks' many end up empty or cut.
double rows_us(bool ragged, int64_t seq_len, double mega)
{
    // a token's latency, or the vector ALU
    return (5.0 + fmax(0.285 * seq_len, 0.57 * mega)) * (ragged ? 0.85 : 1.0);
}

// Sweeping workgroups of `waves` waves; a CU holds 16 waves, or as many workgroups
// as its LDS does.
double sweep_us(int waves, bool ragged, int64_t blocks, int64_t tiles, int64_t seq_len)
{
    const int64_t sub = sweep_tokens(waves), steps = (seq_len + sub * waves - 1) / (sub * waves);
    const int64_t lds = 4 * (waves * (16 * (2 * sub + 4) + 1024 + sub * 16) + tiles * 512);
    const int64_t fit = 163840 / lds, per_cu = fit < 16 / waves ? (fit < 1 ? 1 : fit) : 16 / waves;
    const int64_t slots = 256 * per_cu, rest = blocks % slots;
    auto step = [](int64_t w) { return 3.15 + 0.27 * w; };  // w waves on a CU
    const double rounds = (blocks / slots) * step(per_cu * waves) +
                          (rest ? step(waves * ((rest + 255) / 256)) : 0.0);
    const double body = steps * (0.3 + 0.7 * tiles);
    if (waves == 4)
        return 3.0 + rounds * (0.1 + body) * (ragged ? 0.3 : 0.48);
    if (waves == 8)
        return 3.0 + rounds * (0.08 + body) * (ragged ? 0.69 : 0.92);
    return 3.0 + rounds * (0.19 + body) * (ragged ? 0.82 : 1.03);
}

double chunks_us(bool cut, bool ragged, int64_t tiles, int64_t seq_len, double mega)
{
    const double us = cut ? 41.0 + (tiles > 1 ? 0.555 : 0.4) * mega
                          : 16.5 + fmax(0.35 * seq_len, 0.31 * mega);
    return us * (ragged ? 0.8 : 1.0);
}

// Which evaluation a call takes, and its cut: the one with the least estimate.
// Measured (us, rows | sweep of 4, 8, 16 waves | chunks):
//   64 x 32 x 2560                 48 | 43, 128, 339   | 44
//   8 x 64 x 2560                  26 | 14, 23, 47     | 45
//   16 x 256 x 1024                76 | 35, 34, 42     | 52
//   4 x 512 x 2560                145 | 52, 47, 55     | 66
//   1 x 512 x 1536                128 | 35, 22, 20     | 42
//   1 x 2048 x 1536               552 | 128, 75, 61    | 59
//   1 x 2048 x 5120               579 | 172, 121, 130  | 108
//   64 x 64 x 5120                169 | 149, 288, 717  | 112
//   2 x 509 x 1536, dstate 64     146 | 101, 58, 55    | 82
//   4 x 512 x 2560, dstate 64     246 | 159, 132, 152  | 241
//   8 x 777 x 2560, uneven        179 | 57, 66, 87     | 86
//   64 x 500 x 1024, uneven       268 | 145, 193, 283  | 234
//   1 x 4096 x 1024, dstate 128  1725 | 1405, 783, 714 | 361
// Chunks are as long as leaves about three waves for each of the GPU's 1,024
// SIMDs: every chunk costs its end, its fold and 4 KiB of traffic, and too few
// leave SIMDs idle (1 x 2048 x 5120: 113 us at 2.5 waves a SIMD, 102 at three, 104
// at four, 109 at eight). With context_lengths rows end early and unevenly, and
// shorter chunks fill the gaps (8 x 777 x 2560 with lengths from an eighth up: 135
// us at three, 93 at six, 86 at eight, 87 at ten).
ScanPlan scan_plan(int64_t batch, int64_t dim, int64_t dstate, int64_t ngroups, int64_t seq_len,
                   bool ragged)
{
    ScanPlan q = {};
    const int64_t tiles = (dstate + kStates - 1) / kStates;
    const int64_t blocks = batch * ngroups * ((dim / ngroups + 15) / 16);
    const double mega = 1e-6 * (double)batch * (double)dim * (double)(tiles * kStates) * (double)seq_len;
    int64_t held = 4;  // states that a channel's lanes hold: a power of two
    while (held < dstate)
        held *= 2;
    double best = rows_us(ragged, seq_len, mega * held / (tiles * kStates));
    q.rows = true;
    for (int waves = 4; waves <= 16 && seq_len > 1; waves *= 2) {
        const double us = sweep_us(waves, ragged, blocks, tiles, seq_len);
        if (us < best && launchable(blocks, 64 * waves)) {
            best = us;
            q.rows = false;
            q.sweep = waves;
        }
    }
    q.s.tiles = (int32_t)tiles;
    q.s.per_group = (int32_t)((dim / ngroups + 63) / 64);
    q.s.blocks = (int32_t)(q.s.per_group * ngroups);
    const int64_t waves = batch * q.s.blocks * q.s.tiles, target = (ragged ? 8 : 3) * 1024;
    int64_t chunks = waves * 2 > target ? 1 : target / waves;
    int64_t len = (seq_len + chunks - 1) / chunks;
    len = (len + kBatch - 1) / kBatch * kBatch;
    if (len < 32)
        len = 32;
    chunks = (seq_len + len - 1) / len;
    const __int128 packed = (__int128)batch * seq_len * ngroups * tiles;  // sixteens of B and C
    if (seq_len <= 16 || best <= chunks_us(chunks > 1, ragged, tiles, seq_len, mega) ||
        !launchable(packed, kStates) || !launchable(waves * chunks, 64))
        return q;
    q.rows = false;
    q.sweep = 0;
    q.s.chunk = (int32_t)(len > seq_len ? seq_len : len);
    q.s.chunks = (int32_t)chunks;
    const int most = q.s.tiles <= 4 ? 4 : q.s.tiles <= 8 ? 2 : 1;
    q.s.team = chunks == 1 ? 1 : (chunks == 2 && most > 2) ? 2 : most;
    q.bc_floats = (batch * seq_len * ngroups * q.s.tiles + 1) * (2 * kStates);
    q.start_floats = batch * (chunks + 1) * q.s.blocks * q.s.tiles * (kStates * 64);
    q.sum_floats = batch * (chunks + 1) * q.s.blocks * 64;
    return q;
}

}  // namespace

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
