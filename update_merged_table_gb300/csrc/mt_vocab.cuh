// The losses over a vocabulary: what their files share (mt_vocab.cu: entry points
// and the kernels around the products; mt_vocab_logits.cu: the tiles of logits;
// mt_vocab_sums.cu: the gradients' products).
#pragma once

#include <cuda.h>

#include "mt_parts.cuh"

namespace mt {

// The rows that take part, one after the other: "live" rows below.  Everything is sized for n rows; how many are live is
// known on the device only.
struct LiveRows {
  const int* count;     // [1]
  const int* ids;       // [n][top] a live row's targets in ascending order (top = 1: its target)
  const float* share;   // [n][top] what each of them has of the target distribution
  int top;
};

// The products x W^T of a piece of the vocabulary, as both kernels of logits see them.
struct LogitParams {
  int passes, a_part, b_part, promote, steps;
  int32_t* status;
  LiveRows rows;
  int v0, columns;      // the piece: its first entry of the vocabulary, how many it has
  int kept;             // steps of x (of all parts) that a block keeps, 0: none
  int tiles;            // of 256 columns
  int max_chunks;       // runs of tiles that the statistics have room for
  float scale2;         // scale * log2(e)
  // statistics
  float2* part;         // [2 max_chunks][stride]: per run and team, the largest z and sum of 2^(z - that)
  float* sum_z;         // the same shape: sums of the logits before the scale (smoothing), or NULL
  float* picked;        // [n][top] the logits of the row's targets, before the scale
  size_t stride;
  int* chunks;          // [1] how many runs the statistics were taken in
  // gradient of the logits
  const float4* coef;   // [n] {lse * log2(e), factor of p, what is taken off everywhere, factor of the targets' shares}
  __nv_bfloat16* dz;    // [stride][parts][width]
  int width;            // columns of a part of dz: those of the piece in multiples of 64, zeros behind them
  CUtensorMap map_dz;   // dz in boxes of 64 columns by 32 rows
};
// Steps of 64 columns (of all parts) up to which a block keeps its rows of x.  While dz is written, copies take longer (2950
// clocks against 2000) and the four stages that eight kept steps leave do not hide it: 7373 rows x 100,003 entries x 512,
// statistics 400 us kept and 442 not, dz 606 kept and 543 not.
constexpr int kLogitKept = 8, kGradKept = 6;
cudaError_t launch_logit_stats(const LogitParams& p, const CUtensorMap& a, const CUtensorMap& b, long long row_tiles, bool pair,
                               cudaStream_t s);
cudaError_t launch_logit_grad(const LogitParams& p, int parts, const CUtensorMap& a, const CUtensorMap& b, long long row_tiles, bool pair,
                              cudaStream_t s);

// Terms of a gradient's sum after which it starts anew at the latest.  The tensor core cuts its accumulator off towards zero at
// every 16 of them, by up to 2^-23 of it where all have one sign and size (2^21 such terms: 1.6% lost), by 1e-9 or so where
// signs vary; so this much loses 2^-9 at most, half of what a gradient's own rounding to bf16 may.  Measured without and with
// the cut: 20,000 rows x 300,000 x 64 dx 1572 and 1398 us (more runs fit too), 300,000 x 20,000 x 64 dW 1891 and 2022.
constexpr int kLongest = 1 << 18;

// C = A B.  The tiles that make whole rounds of the blocks have the whole contraction, up to kLongest; that of the rest (all of
// them where there are few, or where it is longer) is cut into runs, each with its own fp32 partial product, so that the last round is a full one too.
struct SumParams {
  int passes, a_part, b_part, promote;  // (fp32: every step brings all parts, so one pass)
  int32_t* status;
  const int* live;      // [1]: rows of C (dx), or the contraction's length (dW)
  int rows;             // rows of C (dW)
  int steps;            // of the contraction (dx)
  int usual;            // steps of a whole piece (dx): by these the runs are chosen, the same ones for every piece
  int columns, ctiles;  // of C
  int max_runs;         // that there is room for
  int* cut;             // [2] the rows of C before those that come in runs, and the runs
  float* part;          // [max_runs][stride][columns]: dx of all rows (one run: the first), dW of the rows behind cut[0]
  size_t stride;
  bool add;             // to what is there
  int reach, reach_part;
  void* out;            // dW [rows][columns]
};
// Columns of a tile of C with this many columns.
inline int sum_width(int64_t columns, bool fp32) { return columns <= 64 ? 64 : columns <= 128 || fp32 ? 128 : 256; }
cudaError_t launch_rows_sum(const SumParams& p, bool fp32, const CUtensorMap& a, const CUtensorMap& b, long long row_tiles, bool pair,
                            cudaStream_t s);
cudaError_t launch_vocab_sum(const SumParams& p, bool fp32, const CUtensorMap& a, const CUtensorMap& b, long long row_tiles, bool pair,
                             cudaStream_t s);

// The statistics and gradients for narrow rows, without a dz in memory (mt_vocab_fused.cu): bf16, up to 128 columns.  Measured, backward
// of 16,384 rows x 50,000 entries, without dz against with: 64 columns 487 against 950 us, 128 604 against 1013, 192 1336
// against 1067; of 2048 x 100,003: 156 / 263, 203 / 281, 361 / 295.
struct FusedParams {
  int32_t* status;
  LiveRows rows;
  int vocab, columns;
  int max_chunks;      // runs of the streamed tiles that there is room for
  int whole;           // dW: kept tiles that go over all streamed tiles, and to `out`
  int* cut;            // [2] the rows of such tiles, and the runs that the others are cut into
  float scale2;
  const float4* coef;
  float* part;         // [max_chunks][stride][columns]: dx of all rows (of a whole tile in the first run), dW of those behind the whole tiles
  size_t stride;
  int reach, reach_part;  // of out's rows and part's
  __nv_bfloat16* out;  // dW
  // statistics: as in LogitParams, kNarrowTeams to a run
  float2* stats;
  float* sum_z;
  float* picked;
};
constexpr int kNarrowTeams = 3;
cudaError_t launch_narrow_stats(const FusedParams& p, const CUtensorMap& x, const CUtensorMap& w, long long units, cudaStream_t s);
constexpr int kFusedColumns = 128, kFusedTile = 128;
cudaError_t launch_fused(bool vocab, const FusedParams& p, const CUtensorMap& x, const CUtensorMap& w, long long units, cudaStream_t s);

}  // namespace mt
