// How a call of the per-channel scan is evaluated, by its sizes alone (ssu_scan.hip
// describes the evaluations). Host code only: it compiles without a GPU's compiler.
#pragma once

#include <math.h>
#include <stdint.h>

#include "ssu_internal.h"

namespace ssu {
namespace {

constexpr int kStates = 16;  // state entries of a lane in the chunk kernels
constexpr int kBatch = 4;    // tokens loaded together

}  // namespace

// Workspace, in floats: packed B | C [batch][seq_len][ngroups][tiles][2][16],
// and a line of 32 zeros; chunk ends [batch][chunks + 1][blocks][tiles][16][64]
// (slot 0 a copy of the pool's state, so that the kernel that writes the pool
// does not read it; slot c + 1 chunk c's end); chunk sums of dt'
// [batch][chunks + 1][blocks][64], slot c + 1 likewise. A block is 64 channels
// of one group.
struct ChunkShape {
    int32_t tiles, per_group, blocks, chunk, chunks;
    int32_t team;  // chunks of one block that share a workgroup: 1, 2 or 4
    int64_t zeros;  // offset of the zero line in bc
    float *bc, *start, *sum;
};

// Tokens of a sweeping wave and step
constexpr int sweep_tokens(int waves) { return waves == 4 ? 8 : 16; }

// How a call is evaluated (scan_plan).
struct ScanPlan {
    bool rows;
    int32_t sweep;  // waves of a sweeping workgroup: 4, 8 or 16; 0: chunks
    ChunkShape s;
    int64_t bc_floats, start_floats, sum_floats;
};

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
    // (INFINITY: the evaluation does not fit one launch)
    const int64_t lanes = held > 16 ? held / 4 : 4, per_wg = 256 / lanes * (seq_len > 1 ? 1 : 2);
    double best = launchable((__int128)batch * ((dim + per_wg - 1) / per_wg), 256)
                      ? rows_us(ragged, seq_len, mega * held / (tiles * kStates))
                      : INFINITY;
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
    const int most = tiles <= 4 ? 4 : tiles <= 8 ? 2 : 1;
    const int team = chunks == 1 ? 1 : (chunks == 2 && most > 2) ? 2 : most;
    const __int128 packed = (__int128)batch * seq_len * ngroups * tiles;  // sixteens of B and C
    if (seq_len <= 16 || best <= chunks_us(chunks > 1, ragged, tiles, seq_len, mega) ||
        !launchable(packed, kStates) ||
        !launchable(batch * q.s.blocks * ((chunks + team - 1) / team), (int)(64 * team * tiles)))
        return q;
    q.rows = false;
    q.sweep = 0;
    q.s.chunk = (int32_t)(len > seq_len ? seq_len : len);
    q.s.chunks = (int32_t)chunks;
    q.s.team = team;
    q.bc_floats = (batch * seq_len * ngroups * q.s.tiles + 1) * (2 * kStates);
    q.start_floats = batch * (chunks + 1) * q.s.blocks * q.s.tiles * (kStates * 64);
    q.sum_floats = batch * (chunks + 1) * q.s.blocks * 64;
    return q;
}

}  // namespace

}  // namespace ssu
