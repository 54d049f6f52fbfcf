// C ABI of the language-model head (log-probabilities and cross entropy from hidden
// states): argument checks, workspace carving and the launch sequence of each
// call, as in api.cpp.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/qlora_nf4.h"
#include "head.h"

using namespace qnf4;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRows = (int64_t)1 << 24, kMaxVocab = (int64_t)1 << 22;
constexpr int64_t kMaxDim = (int64_t)1 << 16, kMaxLd = (int64_t)1 << 22;
// Exponentials that a call keeps at a time: 1 GiB of them, 4096 rows of a vocabulary
// of 128256.  More rows a panel would not make the products faster, fewer would
// leave dW's sums to pass through memory more often.
constexpr int64_t kPanel = (int64_t)1 << 29;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
qlora_status hip_status(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP; }

qlora_status check_sizes(const qlora_head* h) {
  if (!h || h->rows < 0 || h->dim < 1 || h->vocab < 1 || h->ld_hidden < h->dim ||
      h->ld_weight < h->dim)
    return QLORA_ERR_INVALID_ARG;
  if (h->dim % 64 || h->dim > kMaxDim || h->rows >= kMaxRows || h->vocab > kMaxVocab ||
      h->ld_hidden % 8 || h->ld_weight % 8 || h->ld_hidden >= kMaxLd || h->ld_weight >= kMaxLd)
    return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

qlora_status check_head(const qlora_head* h) {
  const qlora_status st = check_sizes(h);
  if (st != QLORA_OK) return st;
  if (!h->weight || !aligned(h->weight, 16)) return QLORA_ERR_INVALID_ARG;
  if (h->rows > 0 && (!h->hidden || !h->labels || !aligned(h->hidden, 16) || !aligned(h->labels, 8)))
    return QLORA_ERR_INVALID_ARG;
  return QLORA_OK;
}

// A gradient of `dim` columns and its row stride; NULL is not asked for.
bool valid_grad(const qlora_head* h, const void* d, int64_t ld) {
  return !d || (aligned(d, 16) && ld >= h->dim && ld % 8 == 0 && ld < kMaxLd &&
                (d != h->hidden || ld == h->ld_hidden || h->rows < 2));
}

int64_t panel_rows(const qlora_head* h) {
  const int tile = head_tile(h->rows, h->vocab);
  const int64_t all = ceil_div(h->rows > 0 ? h->rows : 1, tile) * tile;
  int64_t rows = kPanel / head_cols(h->vocab) / 256 * 256;
  if (rows < 256) rows = 256;
  return rows < all ? rows : all;
}

struct HeadWs {
  size_t h, src, y, n, stat, w, scale, zy, last, lp, part, shift, e, split, rest, acc,
      total;
};
HeadWs head_layout(const qlora_head* h, bool dh, bool dw) {
  HeadWs L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes);
    return at;
  };
  const int64_t panel = panel_rows(h);
  const size_t all = (size_t)(ceil_div(h->rows > 0 ? h->rows : 1, panel) * panel);
  const size_t cols = (size_t)head_cols(h->vocab);
  const bool grad = dh || dw;
  L.h = take(all * h->dim * 2);
  L.src = take(all * 4);
  L.y = take(all * 4);
  L.n = take(8);
  L.stat = take(grad ? all * sizeof(HeadStat) : 0);
  L.w = take(grad ? all * 4 : 0);
  L.scale = take(grad ? all * sizeof(HeadScale) : 0);
  L.zy = take(all * 8);
  L.last = take(dw ? (size_t)h->vocab * 4 : 0);
  L.lp = take(all * 8);
  L.part = take(cols / 128 * panel * sizeof(HeadPart));
  // (also where dW's path does not use it: more gradients need no less)
  L.shift = take(dh ? cols / 128 * panel * 4 : 0);
  L.e = take(grad ? panel * cols * 2 : 0);
  // parts of whichever product's inner index is cut, one after the other
  const int tile = head_tile(h->rows, h->vocab), dim = (int)h->dim;
  size_t split = head_logits_floats(panel, dim, h->vocab, tile);
  if (dh) split = std::max(split, head_dh_floats(panel, dim, h->vocab, tile));
  if (dw) split = std::max(split, head_dw_floats(panel, dim, h->vocab));
  L.split = take(split * 4);
  L.rest = take(dw ? (size_t)head_slots(panel, h->vocab) * h->dim * 4 : 0);
  L.acc = take(dw && h->rows > panel ? (size_t)h->vocab * h->dim * 4 : 0);
  L.total = off;
  return L;
}

template <typename T>
T* at(void* ws, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(ws) + off); }

HeadPanel panel(const qlora_head* h, void* ws, const HeadWs& L, bool dw) {
  HeadPanel p;
  p.r = HeadRows{at<uint16_t>(ws, L.h), at<int32_t>(ws, L.src), at<int32_t>(ws, L.y),
                 at<int32_t>(ws, L.n), at<HeadStat>(ws, L.stat), at<float>(ws, L.w),
                 at<HeadScale>(ws, L.scale), at<double>(ws, L.zy), at<int32_t>(ws, L.last)};
  p.row0 = 0;
  p.rows = (int)panel_rows(h);
  p.dim = (int)h->dim;
  p.weight = h->weight;
  p.ldw = h->ld_weight;
  p.vocab = h->vocab;
  p.part = at<HeadPart>(ws, L.part);
  p.want_last = dw;
  p.shift = at<uint32_t>(ws, L.shift);
  p.splits = head_dh_splits(p.rows, p.dim, p.vocab, head_tile(h->rows, h->vocab));
  p.e = at<uint16_t>(ws, L.e);
  return p;
}

HeadPackArgs pack_args(const qlora_head* h, const HeadPanel& p) {
  HeadPackArgs a = {};
  a.hidden = h->hidden;
  a.ldh = h->ld_hidden;
  a.rows = h->rows;
  a.dim = (int)h->dim;
  a.vocab = h->vocab;
  a.weight = h->weight;
  a.ldw = h->ld_weight;
  a.labels = h->labels;
  a.to = p.r;
  a.panel = p.rows;
  a.tile = head_tile(h->rows, h->vocab);
  return a;
}

// dh and dW of a panel whose e holds dz, or (pow, without dW) the powers of two
hipError_t panel_grads(const qlora_head* h, const HeadPanel& p, void* ws, const HeadWs& L, int tile,
                       int pow, uint16_t* dh, int64_t ldd, uint16_t* dw, int64_t ldo, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (dh) e = launch_head_dh(p, tile, pow, at<float>(ws, L.split), dh, ldd, s);
  if (e == hipSuccess && dw) e = launch_head_rest(p, at<float>(ws, L.rest), s);
  if (e == hipSuccess && dw)
    e = launch_head_dw(p, at<float>(ws, L.rest), at<float>(ws, L.split),
                       h->rows > p.rows ? at<float>(ws, L.acc) : nullptr, p.row0 == 0,
                       p.row0 + p.rows >= h->rows, dw, ldo, s);
  return e;
}

bool opt4(const void* p) { return aligned(p, 4); }   // NULL passes

}  // namespace

extern "C" {

size_t qlora_head_workspace_bytes(const qlora_head* h, int32_t grads) {
  if (check_sizes(h) != QLORA_OK || (grads & ~(QLORA_HEAD_DHIDDEN | QLORA_HEAD_DWEIGHT))) return 0;
  return head_layout(h, grads & QLORA_HEAD_DHIDDEN, grads & QLORA_HEAD_DWEIGHT).total;
}

qlora_status qlora_head_logprobs(const qlora_head* h, float* logp, float* stats, void* ws,
                                 size_t ws_bytes, void* stream) {
  const qlora_status st = check_head(h);
  if (st != QLORA_OK) return st;
  if ((h->rows > 0 && !logp) || !opt4(logp) || !opt4(stats)) return QLORA_ERR_INVALID_ARG;
  if (h->rows == 0) return QLORA_OK;
  const HeadWs L = head_layout(h, false, false);
  if (!ws || ws_bytes < L.total || !aligned(ws, kAlign)) return QLORA_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  HeadPanel p = panel(h, ws, L, false);
  HeadPackArgs a = pack_args(h, p);
  a.logp = logp;
  a.stat_out = reinterpret_cast<HeadStat*>(stats);
  const int tile = head_tile(h->rows, h->vocab);
  hipError_t e = launch_head_pack(a, s);
  for (; e == hipSuccess && p.row0 < h->rows; p.row0 += p.rows) {
    e = launch_head_logits(p, tile, HEAD_STATS, at<float>(ws, L.split), s);
    if (e == hipSuccess)
      e = launch_head_join(p, HEAD_SCORE, 0, nullptr, logp, a.stat_out, s);
  }
  return hip_status(e);
}

qlora_status qlora_head_logprobs_bwd(const qlora_head* h, const float* stats, const float* w,
                                     const float* grad_scale, qlora_bf16* dhidden, int64_t ldd,
                                     qlora_bf16* dweight, int64_t ldo, void* ws, size_t ws_bytes,
                                     void* stream) {
  const qlora_status st = check_head(h);
  if (st != QLORA_OK) return st;
  if (!opt4(stats) || !opt4(w) || !opt4(grad_scale) || !valid_grad(h, dhidden, ldd) ||
      !valid_grad(h, dweight, ldo) || (!dhidden && !dweight && h->rows > 0) ||
      (h->rows > 0 && (!stats || !w)))
    return QLORA_ERR_INVALID_ARG;
  if (h->rows == 0 && !dweight) return QLORA_OK;
  const HeadWs L = head_layout(h, dhidden, dweight);
  if (!ws || ws_bytes < L.total || !aligned(ws, kAlign)) return QLORA_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  HeadPanel p = panel(h, ws, L, dweight);
  HeadPackArgs a = pack_args(h, p);
  a.weight = nullptr;   // (the statistics are the caller's)
  a.w = w;
  a.w_scale = grad_scale;
  a.stat = reinterpret_cast<const HeadStat*>(stats);
  a.dh = dhidden;
  a.ldd = ldd;
  a.pad = dweight != nullptr;
  const int tile = head_tile(h->rows, h->vocab);
  hipError_t e = launch_head_pack(a, s);
  do {
    if (e == hipSuccess) e = launch_head_logits(p, tile, HEAD_DZ, at<float>(ws, L.split), s);
    if (e == hipSuccess) e = panel_grads(h, p, ws, L, tile, 0, dhidden, ldd, dweight, ldo, s);
    p.row0 += p.rows;
  } while (e == hipSuccess && p.row0 < h->rows);
  return hip_status(e);
}

qlora_status qlora_head_cross_entropy(const qlora_head* h, int32_t reduction, float* loss,
                                      float* logp, qlora_bf16* dhidden, int64_t ldd,
                                      qlora_bf16* dweight, int64_t ldo, void* ws, size_t ws_bytes,
                                      void* stream) {
  const qlora_status st = check_head(h);
  if (st != QLORA_OK) return st;
  if (!loss || !opt4(loss) || !opt4(logp) || !valid_grad(h, dhidden, ldd) ||
      !valid_grad(h, dweight, ldo) ||
      (reduction != QLORA_HEAD_MEAN && reduction != QLORA_HEAD_SUM))
    return QLORA_ERR_INVALID_ARG;
  const HeadWs L = head_layout(h, dhidden, dweight);
  if (!ws || ws_bytes < L.total || !aligned(ws, kAlign)) return QLORA_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  HeadPanel p = panel(h, ws, L, dweight);
  HeadPackArgs a = pack_args(h, p);
  a.logp = logp;
  a.dh = dhidden;
  a.ldd = ldd;
  a.pad = dweight != nullptr;
  const int tile = head_tile(h->rows, h->vocab), mean = reduction == QLORA_HEAD_MEAN;
  const bool grad = dhidden || dweight, pow = grad && !dweight;
  hipError_t e = launch_head_pack(a, s);
  do {
    if (e == hipSuccess)
      e = launch_head_logits(p, tile, pow ? HEAD_POW : grad ? HEAD_EXP : HEAD_STATS,
                             at<float>(ws, L.split), s);
    if (e == hipSuccess)
      e = launch_head_join(p, !grad ? HEAD_LOSS : mean ? HEAD_GRAD_MEAN : HEAD_GRAD_SUM,
                           pow, at<double>(ws, L.lp), logp, nullptr, s);
    if (e == hipSuccess && dweight) e = launch_head_dz(p, s);
    if (e == hipSuccess && grad) e = panel_grads(h, p, ws, L, tile, pow, dhidden, ldd, dweight, ldo, s);
    p.row0 += p.rows;
  } while (e == hipSuccess && p.row0 < h->rows);
  if (e == hipSuccess) e = launch_head_loss(p.r.n, at<double>(ws, L.lp), mean, loss, s);
  return hip_status(e);
}

}  // extern "C"
