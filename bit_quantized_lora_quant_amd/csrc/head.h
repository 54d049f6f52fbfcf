// Internal launcher interface of the language-model head: log-probabilities and
// cross entropy straight from hidden states.
#pragma once

#include "launch.h"

namespace qnf4 {

// What the forward leaves of a row for its gradient: log sum_v exp(z_v), and
// 1 - p of the target (what is left beside a nearly certain target, which
// 1 - exp(logp) would not have).
struct HeadStat {
  float lse, rest;
};
// A slice's largest logit m and, with M = ceil(m log2 e), a whole number, its sum of
// 2^(z log2 e - M), the target left out of both.
struct HeadPart {
  float m, s;
};
// A row's gradient: the largest m of its slices, whose M is R; f and c with
// dz_v = f 2^(z_v log2 e - R), at the target c = w (1 - p).  (The backward: c alone.)
struct HeadScale {
  float m, f, c;
};

// Rows with a target, packed: hidden [up to a tile's rows][D], their source rows and
// labels (-1: past the vocabulary) and, for the backward, lse / rest / weight.
struct HeadRows {
  uint16_t* h;
  int32_t* src;
  int32_t* y;
  int32_t* n;         // [2] how many, and the slices of dh in a panel they do not fill
  HeadStat* stat;
  float* w;
  HeadScale* scale;
  double* zy;         // the target's logit
  int32_t* last;      // [vocab] the last packed row with that target, -1 none (for dW)
};

struct HeadPackArgs {
  const uint16_t* hidden;
  int64_t ldh, rows;
  int dim;
  int64_t vocab;
  const uint16_t* weight;  // nullable: no target's logit
  int64_t ldw;
  const int64_t* labels;
  const float* w;          // nullable: rows of weight 0 count as without target
  const float* w_scale;    // nullable, [1]
  const HeadStat* stat;    // with w
  HeadRows to;
  int panel, tile;         // rows of a panel and of a tile
  int pad;                 // for dW: zero rows behind the last, and to.last
  // rows without a target, each nullable
  float* logp;
  HeadStat* stat_out;
  uint16_t* dh;
  int64_t ldd;
};
hipError_t launch_head_pack(const HeadPackArgs& a, hipStream_t s);

// One panel of packed rows [row0, row0 + rows) (as many as there are), rows a
// multiple of the tile.
struct HeadPanel {
  HeadRows r;
  int64_t row0;
  int rows;
  int dim;
  const uint16_t* weight;
  int64_t ldw, vocab;
  HeadPart* part;      // [vocab tiles * 2][rows]
  uint32_t* shift;     // [vocab tiles * 2][rows] R - M, in both halves as bf16's exponent
  int splits;          // slices of dh in a full panel
  int want_last;       // r.last is needed (dW)
  uint16_t* e;         // [rows][head_cols(vocab)] exponents in 16 bits, then dz (bf16)
};
// Columns of a panel's row.
__host__ __device__ inline int64_t head_cols(int64_t vocab) { return ceil_div(vocab, 256) * 256; }
int head_dh_splits(int64_t rows, int dim, int64_t vocab, int tile);
// Rows of tokens per workgroup tile (64, 128 or 256) of a call.
int head_tile(int64_t rows, int64_t vocab);

// HEAD_STATS: part; HEAD_EXP: part and e's exponents; HEAD_DZ: dz from r.stat and r.w;
// HEAD_POW: as HEAD_EXP with powers in bf16, which dh takes as they are
enum { HEAD_STATS = 0, HEAD_EXP = 1, HEAD_DZ = 2, HEAD_POW = 3 };
// part: head_logits_floats floats (of partial logits, where the inner index is cut)
size_t head_logits_floats(int64_t rows, int dim, int64_t vocab, int tile);
hipError_t launch_head_logits(const HeadPanel& p, int tile, int mode, float* part, hipStream_t s);
// Joins the slices: logp and stat of the rows (nullable, by source row).
// From HEAD_LOSS on the packed rows' logp in lp; with HEAD_GRAD_* also r.scale for
// w = -1 (sum) or -1 / n (mean), and p.shift where `shift`.
enum { HEAD_SCORE = 0, HEAD_LOSS = 1, HEAD_GRAD_SUM = 2, HEAD_GRAD_MEAN = 3 };
hipError_t launch_head_join(const HeadPanel& p, int kind, int shift, double* lp, float* logp,
                            HeadStat* stat, hipStream_t s);
hipError_t launch_head_loss(const int32_t* n, const double* lp, int mean, float* loss,
                            hipStream_t s);
// e -> dz in place
hipError_t launch_head_dz(const HeadPanel& p, hipStream_t s);
// dh = dz . W by source row, from e's dz, or (pow) from HEAD_POW's e, p.shift and
// r.scale; part: head_dh_floats floats
size_t head_dh_floats(int64_t rows, int dim, int64_t vocab, int tile);
hipError_t launch_head_dh(const HeadPanel& p, int tile, int pow, float* part, uint16_t* dh, int64_t ldd,
                          hipStream_t s);
// What rounding the targets' dz leaves of dW, in float32: rest[head_slot] = sum over the
// panel's rows with that target of (c - bf16(c)) h.
__host__ __device__ inline int64_t head_slots(int64_t rows, int64_t vocab) {
  return rows < vocab ? rows : vocab;
}
hipError_t launch_head_rest(const HeadPanel& p, float* rest, hipStream_t s);
// dw = dz^T . h + rest (bf16, row stride ldo), or with acc [vocab][dim] over several
// panels: added to it (stored where first), and only the last writes dw.
// part: head_dw_floats floats
size_t head_dw_floats(int64_t rows, int dim, int64_t vocab);
hipError_t launch_head_dw(const HeadPanel& p, const float* rest, float* part, float* acc, int first,
                          int last, uint16_t* dw, int64_t ldo, hipStream_t s);

}  // namespace qnf4
