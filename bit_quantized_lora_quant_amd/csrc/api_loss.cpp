// C ABI of the losses on packed logits: argument checks, workspace carving and
// the launch sequence of each call, as in api.cpp.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/qlora_nf4.h"
#include "loss.h"

using namespace qnf4;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRows = (int64_t)1 << 24, kMaxVocab = (int64_t)1 << 30;
constexpr int32_t kMaxSequences = 1 << 22;   // a workgroup of 512 threads each, in one dimension

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t esize(const qlora_logits* z) { return z->dtype == QLORA_BF16 ? 2 : 4; }

qlora_status hip_status(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP; }

qlora_status check_sizes(const qlora_logits* z) {
  if (!z || (z->dtype != QLORA_F32 && z->dtype != QLORA_BF16) || z->reserved != 0)
    return QLORA_ERR_INVALID_ARG;
  if (z->rows < 0 || z->vocab < 1 || z->ld < z->vocab) return QLORA_ERR_INVALID_ARG;
  if (z->rows >= kMaxRows || z->vocab >= kMaxVocab || z->ld >= kMaxVocab)
    return QLORA_ERR_UNSUPPORTED;
  // the gradient launch's workgroups of 256 threads, in one grid dimension
  if (z->rows * row_grad_slices(z->vocab, z->dtype == QLORA_BF16) >= kMaxRows)
    return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

// (the statistics launch has a workgroup for each of both)
bool too_many(const qlora_logits* z, int64_t sequences) {
  return sequences >= kMaxSequences || z->rows + sequences >= kMaxRows;
}

qlora_status check_logits(const qlora_logits* z) {
  const qlora_status st = check_sizes(z);
  if (st != QLORA_OK) return st;
  if (z->rows > 0 && (!z->data || !z->labels || !aligned(z->data, esize(z)) ||
                      !aligned(z->labels, 8)))
    return QLORA_ERR_INVALID_ARG;
  return QLORA_OK;
}

bool valid_grad(const qlora_logits* z, const void* dz, int64_t ldd) {
  if (!aligned(dz, esize(z)) || ldd < z->vocab || ldd >= kMaxVocab) return false;
  return dz != z->data || ldd == z->ld;
}

LogitsView view(const qlora_logits* z, const int32_t* cu, int32_t nseq) {
  return LogitsView{z->data, z->dtype == QLORA_BF16, z->rows, z->vocab, z->ld, z->labels, cu, nseq};
}

// Scratch of one call: what the caller does not take of the rows' outputs,
// their slices, the sums of the sequences and the counter.
struct LossWs {
  size_t logp, stats, w, zy, part, count, seq, list, sums, ticket, total;
};
LossWs loss_layout(const qlora_logits* z, int32_t sequences) {
  LossWs L;
  size_t off = 0;
  const size_t rows = (size_t)z->rows, seqs = (size_t)sequences;
  const int slices = row_slices(view(z, nullptr, 0));
  L.logp = off;   off = align_up(off + rows * sizeof(float));
  L.stats = off;  off = align_up(off + rows * sizeof(MaxSum));
  L.w = off;      off = align_up(off + rows * sizeof(float));
  L.zy = off;     off = align_up(off + rows * sizeof(float));
  L.part = off;   off = align_up(off + (slices > 1 ? rows * slices : 0) * sizeof(MaxSum));
  L.count = off;  off = align_up(off + seqs * sizeof(int));
  L.seq = off;    off = align_up(off + (seqs > 0 ? rows : 0) * sizeof(int));
  L.list = off;   off = align_up(off + (seqs > 0 ? rows + 1 : 0) * sizeof(int));
  L.sums = off;   off = align_up(off + seqs * 3 * sizeof(double));
  L.ticket = off; off = align_up(off + sizeof(uint32_t));
  L.total = off;
  return L;
}

template <typename T>
T* at(void* ws, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(ws) + off); }

RowOut row_out(void* ws, const LossWs& L, float* logp, float* stats, float* w) {
  return RowOut{logp ? logp : at<float>(ws, L.logp),
                stats ? reinterpret_cast<MaxSum*>(stats) : at<MaxSum>(ws, L.stats),
                w ? w : at<float>(ws, L.w), at<float>(ws, L.zy), at<MaxSum>(ws, L.part),
                at<uint32_t>(ws, L.ticket)};
}

bool opt4(const void* p) { return aligned(p, 4); }   // NULL passes

}  // namespace

extern "C" {

size_t qlora_loss_workspace_bytes(const qlora_logits* z, int32_t sequences) {
  if (check_sizes(z) != QLORA_OK || sequences < 0 || too_many(z, sequences)) return 0;
  return loss_layout(z, sequences).total;
}

qlora_status qlora_token_logprobs(const qlora_logits* z, float* logp, float* stats, void* ws,
                                  size_t ws_bytes, void* stream) {
  const qlora_status st = check_logits(z);
  if (st != QLORA_OK) return st;
  if ((z->rows > 0 && !logp) || !opt4(logp) || !opt4(stats)) return QLORA_ERR_INVALID_ARG;
  if (z->rows == 0) return QLORA_OK;
  const LossWs L = loss_layout(z, 0);
  if (!ws || ws_bytes < L.total || !aligned(ws, kAlign)) return QLORA_ERR_WORKSPACE;
  return hip_status(launch_row_logp(view(z, nullptr, 0), row_out(ws, L, logp, stats, nullptr),
                                    static_cast<hipStream_t>(stream)));
}

qlora_status qlora_token_logprobs_bwd(const qlora_logits* z, const float* stats, const float* w,
                                      const float* grad_scale, void* dlogits, int64_t ldd,
                                      void* stream) {
  const qlora_status st = check_logits(z);
  if (st != QLORA_OK) return st;
  if (!opt4(stats) || !opt4(w) || !opt4(grad_scale) || !valid_grad(z, dlogits, ldd))
    return QLORA_ERR_INVALID_ARG;
  if (z->rows == 0) return QLORA_OK;
  if (!stats || !w || !dlogits) return QLORA_ERR_INVALID_ARG;
  return hip_status(launch_row_grad(view(z, nullptr, 0),
                                    reinterpret_cast<const MaxSum*>(stats), w, grad_scale, dlogits,
                                    ldd, static_cast<hipStream_t>(stream)));
}

qlora_status qlora_preference_loss(const qlora_logits* z, int32_t pairs, const int32_t* cu_seqlens,
                                   const float* ref_logp, const qlora_preference_params* h,
                                   float* loss, float* seq_logp, float* rewards, float* logp,
                                   float* stats, float* w, void* dlogits, int64_t ldd, void* ws,
                                   size_t ws_bytes, void* stream) {
  const qlora_status st = check_logits(z);
  if (st != QLORA_OK) return st;
  if (pairs < 1 || !cu_seqlens || !opt4(cu_seqlens) || !h || !loss || !opt4(loss))
    return QLORA_ERR_INVALID_ARG;
  if (!opt4(ref_logp) || !opt4(seq_logp) || !opt4(rewards) || !opt4(logp) || !opt4(stats) ||
      !opt4(w) || (dlogits && !valid_grad(z, dlogits, ldd)))
    return QLORA_ERR_INVALID_ARG;
  if (!(h->beta > 0) || !std::isfinite(h->beta) ||
      !(h->label_smoothing >= 0 && h->label_smoothing <= 0.5) || h->kind < QLORA_PREF_SIGMOID ||
      h->kind > QLORA_PREF_IPO || (h->kind != QLORA_PREF_SIGMOID && h->label_smoothing != 0) ||
      (h->length_mean != 0 && h->length_mean != 1))
    return QLORA_ERR_INVALID_ARG;
  if (too_many(z, 2 * (int64_t)pairs)) return QLORA_ERR_UNSUPPORTED;
  const LossWs L = loss_layout(z, 2 * pairs);
  if (!ws || ws_bytes < L.total || !aligned(ws, kAlign)) return QLORA_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const LogitsView v = view(z, cu_seqlens, 2 * pairs);
  const RowOut o = row_out(ws, L, logp, stats, w);
  const PreferenceArgs a{pairs,          ref_logp, h->beta,  h->label_smoothing, h->kind,
                         h->length_mean, loss,     seq_logp, rewards,            at<double>(ws, L.sums)};
  hipError_t e = launch_preference(v, o, a, s);
  if (e == hipSuccess && dlogits) e = launch_row_grad(v, o.stats, o.w, nullptr, dlogits, ldd, s);
  return hip_status(e);
}

qlora_status qlora_policy_loss(const qlora_logits* z, int32_t sequences,
                               const int32_t* cu_seqlens, const float* advantages,
                               const float* old_logp, const float* ref_logp,
                               const qlora_policy_params* h, float* out, float* logp,
                               float* stats, float* w, void* dlogits, int64_t ldd, void* ws,
                               size_t ws_bytes, void* stream) {
  const qlora_status st = check_logits(z);
  if (st != QLORA_OK) return st;
  if (sequences < 1 || !cu_seqlens || !opt4(cu_seqlens) || !advantages || !opt4(advantages) ||
      !h || !out || !opt4(out))
    return QLORA_ERR_INVALID_ARG;
  if (!opt4(old_logp) || !opt4(ref_logp) || !opt4(logp) || !opt4(stats) || !opt4(w) ||
      (dlogits && !valid_grad(z, dlogits, ldd)))
    return QLORA_ERR_INVALID_ARG;
  if (!(h->clip_low >= 0 && h->clip_low <= 1) || !(h->clip_high >= 0) ||
      !std::isfinite(h->clip_high) || !(h->kl_coef >= 0) || !std::isfinite(h->kl_coef) ||
      (h->kl_coef > 0 && !ref_logp) ||
      (h->reduction != QLORA_POLICY_TOKEN && h->reduction != QLORA_POLICY_SEQUENCE) ||
      (h->token_advantages != 0 && h->token_advantages != 1))
    return QLORA_ERR_INVALID_ARG;
  if (too_many(z, sequences)) return QLORA_ERR_UNSUPPORTED;
  const LossWs L = loss_layout(z, sequences);
  if (!ws || ws_bytes < L.total || !aligned(ws, kAlign)) return QLORA_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const LogitsView v = view(z, cu_seqlens, sequences);
  const RowOut o = row_out(ws, L, logp, stats, w);
  const PolicyArgs a{advantages,          old_logp, ref_logp, 1 - h->clip_low, 1 + h->clip_high,
                     h->kl_coef,          h->reduction, h->token_advantages, out,
                     at<int>(ws, L.count), at<int>(ws, L.seq), at<int>(ws, L.list),
                     at<double>(ws, L.sums)};
  return hip_status(launch_policy(v, o, a, dlogits, ldd, s));
}

}  // extern "C"
