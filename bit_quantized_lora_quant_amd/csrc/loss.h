// Internal launcher interface of the losses on packed logits.
#pragma once

#include "launch.h"

namespace qnf4 {

// Logits [rows, vocab] (row stride ld) with their targets; cu (nullable): rows
// outside [cu[0], cu[nseq]) have none.
struct LogitsView {
  const void* z;
  int bf16;
  int64_t rows, vocab, ld;
  const int64_t* labels;
  const int32_t* cu;
  int nseq;
};

// Maximum m and sum of exp(z - m) of a row, or of a slice of one.
struct MaxSum {
  float m, s;
};

// What a loss writes for each row (logp, stats, w = dLoss / dlogp) and its
// scratch: the target's logit (the logits may be overwritten by the gradient
// before the sums), the slices' statistics [rows][row_slices] and a counter.
struct RowOut {
  float* logp;
  MaxSum* stats;
  float* w;
  float* zy;
  MaxSum* part;
  uint32_t* ticket;
};

struct PreferenceArgs {
  int pairs;
  const float* ref;       // nullable
  double beta, smooth;
  int kind, length_mean;
  float* loss;            // [1]
  float* seq_logp;        // nullable, [2 pairs]
  float* rewards;         // nullable, [2 pairs]
  double* pair_loss;      // scratch [pairs]
};

struct PolicyArgs {
  const float* adv;
  const float* old_logp;  // nullable
  const float* ref;       // nullable
  double lo, hi, kl_coef; // clamp bounds 1 - clip_low, 1 + clip_high
  int reduction, token_adv;
  float* out;             // [3]
  int* count;             // scratch [nseq]: targets of each sequence
  int* seq;               // scratch [rows]: sequence of each row in one
  int* list;              // scratch [rows + 1]: the rows with a target, their number last
  double* sums;           // scratch [nseq][3]: loss, kl, clipped
};

// Slices of a row in the statistics launch.
int row_slices(const LogitsView& v);
// Workgroups of a row in the gradient launch.
int64_t row_grad_slices(int64_t vocab, int bf16);
// stats and logp of every row with a target
hipError_t launch_row_logp(const LogitsView& v, const RowOut& o, hipStream_t s);
hipError_t launch_preference(const LogitsView& v, const RowOut& o, const PreferenceArgs& a,
                             hipStream_t s);
// with the gradient in dz (nullable, row stride ldd)
hipError_t launch_policy(const LogitsView& v, const RowOut& o, const PolicyArgs& a, void* dz,
                         int64_t ldd, hipStream_t s);
// dlogits = g w (1[y] - exp(z - m) / sum), row stride ldd
hipError_t launch_row_grad(const LogitsView& v, const MaxSum* stats, const float* w,
                           const float* g, void* dz, int64_t ldd, hipStream_t s);

}  // namespace qnf4
