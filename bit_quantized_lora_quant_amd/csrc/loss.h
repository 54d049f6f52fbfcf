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

// What a loss writes for each row: logp, stats (m, sum) and w = dLoss / dlogp.
struct RowOut {
  float* logp;
  float* stats;
  float* w;
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
  double* sums;           // scratch [nseq][4]: loss, kl, clipped, targets
};

hipError_t launch_row_stats(const LogitsView& v, const RowOut& o, hipStream_t s);
hipError_t launch_preference(const LogitsView& v, const RowOut& o, const PreferenceArgs& a,
                             hipStream_t s);
hipError_t launch_policy(const LogitsView& v, const RowOut& o, const PolicyArgs& a, hipStream_t s);
// dlogits = g w (1[y] - exp(z - m) / sum), row stride ldd
hipError_t launch_row_grad(const LogitsView& v, const float* stats, const float* w,
                           const float* g, void* dz, int64_t ldd, hipStream_t s);

}  // namespace qnf4
