// C ABI of the orthogonalised update: argument checks, workspace carving and the
// launch sequence of each call, as in api.cpp.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/qlora_nf4.h"
#include "muon.h"

using namespace qnf4;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxIndex = (int64_t)1 << 30;    // rows, columns and strides
constexpr int64_t kMaxGroups256 = (int64_t)1 << 24;   // workgroups of 256 threads in a grid

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
qlora_status hip_status(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP; }

bool valid_type(qlora_dtype t) { return t == QLORA_F32 || t == QLORA_BF16; }
size_t esize(qlora_dtype t) { return t == QLORA_BF16 ? 2 : 4; }

qlora_status check_shape(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return QLORA_ERR_INVALID_ARG;
  if (rows >= kMaxIndex || cols >= kMaxIndex) return QLORA_ERR_UNSUPPORTED;
  if ((rows < cols ? rows : cols) > kMaxRank) return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}
// a matrix's pointer (not NULL) and row stride
bool valid_matrix(const void* p, size_t size, int64_t ld, int64_t cols) {
  return p && aligned(p, size) && ld >= cols && ld < kMaxIndex;
}

bool valid_ns(const qlora_newton_schulz* n) {
  return n && n->steps >= 1 && n->steps <= 32 && n->reserved == 0 && std::isfinite(n->a) &&
         std::isfinite(n->b) && std::isfinite(n->c) && n->eps > 0 && std::isfinite(n->eps);
}

// The call's tensors as the kernels see them, one at a time (`get(i)` fills shape,
// pointers and strides); workgroups, parts and polynomials follow one another.
struct Sizes {
  int64_t total = 0;                    // elements
  int64_t count = 0, wgs = 0, chunks = 0, part = 0, q = 0;
  int64_t longest = 0;                  // chunks of a tensor
  uint32_t ranks = 0;                   // bit sp / 16 of each padded short side
};
bool empty(const MuonTensor& t) { return t.rows == 0 || t.cols == 0; }
void place(MuonTensor& t, Sizes& z) {
  const int64_t s = t.rows < t.cols ? t.rows : t.cols, n = t.rows < t.cols ? t.cols : t.rows;
  const int sp = muon_pad((int)s);
  t.slice = muon_slice(sp, z.total);
  t.wg = (int32_t)z.wgs;
  t.chunk = (int32_t)z.chunks;
  t.part = (uint32_t)z.part;
  t.q = (uint32_t)z.q;
  const int64_t wgs = ceil_div(n, t.slice);
  z.count += 1;
  z.wgs += wgs;
  z.chunks += ceil_div(n, muon_chunk(sp));
  z.longest = std::max(z.longest, ceil_div(n, muon_chunk(sp)));
  z.part += wgs * muon_tiles(sp);
  z.q += sp * sp / 256;
  z.ranks |= 1u << (sp / 16);
}
template <typename Get>
Sizes sizes(int32_t count, Get get) {
  Sizes z;
  for (int32_t i = 0; i < count; ++i) {
    const MuonTensor t = get(i);
    z.total += (int64_t)t.rows * t.cols;
  }
  for (int32_t i = 0; i < count; ++i) {
    MuonTensor t = get(i);
    if (!empty(t)) place(t, z);
  }
  return z;
}
bool fits(const Sizes& z) {
  const int64_t most = (int64_t)1 << 32;
  return z.chunks < kMaxGroups256 && z.count < 65536 && z.part < most && z.q < most;
}

struct MuonWs {
  size_t t, owner, owner_wg, part, q, total;
};
MuonWs muon_layout(const Sizes& z) {
  MuonWs L;
  size_t off = 0;
  L.t = off;      off = align_up(off + z.count * sizeof(MuonTensor));
  L.owner = off;  off = align_up(off + z.chunks * sizeof(int32_t));
  L.owner_wg = off;
  off = align_up(off + z.wgs * sizeof(int32_t));
  L.part = off;   off = align_up(off + z.part * 256 * sizeof(double));
  L.q = off;      off = align_up(off + z.q * 256 * sizeof(double));
  L.total = off;
  return L;
}

template <typename Get>
qlora_status run(int32_t count, Get get, const MuonHyper& h, void* ws, size_t ws_bytes,
                 hipStream_t st) {
  const Sizes z = sizes(count, get);
  if (!fits(z)) return QLORA_ERR_UNSUPPORTED;
  if (z.count == 0) return QLORA_OK;
  const MuonWs L = muon_layout(z);
  if (!ws || ws_bytes < L.total || !aligned(ws, kAlign)) return QLORA_ERR_WORKSPACE;
  char* base = static_cast<char*>(ws);
  const MuonScratch s{reinterpret_cast<MuonTensor*>(base + L.t),
                      reinterpret_cast<int32_t*>(base + L.owner),
                      reinterpret_cast<int32_t*>(base + L.owner_wg),
                      reinterpret_cast<double*>(base + L.part),
                      reinterpret_cast<double*>(base + L.q)};
  // one batch travels in the first launch's arguments, more through the table
  const bool whole = z.count <= kMuonBatch;
  const bool small = whole && z.longest <= kMuonSmall && z.ranks < 1u << (64 / 16);
  Sizes at;
  at.total = z.total;
  MuonBatch b;
  hipError_t e = hipSuccess;
  for (int32_t i = 0; i < count && e == hipSuccess;) {
    b.count = 0;
    b.first = (int)at.count;
    for (; i < count && b.count < kMuonBatch; ++i) {
      MuonTensor t = get(i);
      if (empty(t)) continue;
      place(t, at);
      b.t[b.count++] = t;
    }
    if (whole) i = count;   // (what is left is empty)
    else if (b.count > 0) e = launch_muon_table(b, s, st);
  }
  // (the first launches of all ranks write the table that the others read)
  auto each = [&](auto launch) {
    for (int sp = 16; sp <= kMaxRank && e == hipSuccess; sp *= 2)
      if (z.ranks >> (sp / 16) & 1) e = launch(sp);
  };
  if (small) {
    each([&](int sp) { return launch_muon_small(b, sp, h, st); });
    return hip_status(e);
  }
  each([&](int sp) { return launch_muon_gram(whole ? &b : nullptr, sp, (int)z.wgs, h, s, st); });
  each([&](int sp) { return launch_muon_poly((int)z.count, sp, h, s, st); });
  each([&](int sp) { return launch_muon_apply(sp, (int)z.chunks, h, s, st); });
  return hip_status(e);
}

MuonTensor shape_of(int64_t rows, int64_t cols) {
  MuonTensor t = {};
  t.rows = (int32_t)rows;
  t.cols = (int32_t)cols;
  return t;
}

}  // namespace

extern "C" {

size_t qlora_muon_workspace_bytes(const int64_t* rows, const int64_t* cols, int32_t count) {
  if (count < 0 || (count > 0 && (!rows || !cols))) return 0;
  for (int32_t i = 0; i < count; ++i)
    if (check_shape(rows[i], cols[i]) != QLORA_OK) return 0;
  const Sizes z = sizes(count, [&](int32_t i) { return shape_of(rows[i], cols[i]); });
  return fits(z) ? muon_layout(z).total : 0;
}

qlora_status qlora_orthogonalize(const qlora_newton_schulz* ns, const qlora_ortho_matrix* m,
                                 int32_t count, void* ws, size_t ws_bytes, void* stream) {
  if (!valid_ns(ns) || count < 0 || (count > 0 && !m)) return QLORA_ERR_INVALID_ARG;
  for (int32_t i = 0; i < count; ++i) {
    if (!valid_type(m[i].dtype) || m[i].reserved != 0) return QLORA_ERR_INVALID_ARG;
    const qlora_status st = check_shape(m[i].rows, m[i].cols);
    if (st != QLORA_OK) return st;
    if (m[i].rows == 0 || m[i].cols == 0) continue;
    const size_t es = esize(m[i].dtype);
    if (!valid_matrix(m[i].in, es, m[i].ld_in, m[i].cols) ||
        !valid_matrix(m[i].out, es, m[i].ld_out, m[i].cols) ||
        (m[i].in == m[i].out && m[i].ld_in != m[i].ld_out))
      return QLORA_ERR_INVALID_ARG;
  }
  MuonHyper h = {};
  h.steps = ns->steps;
  h.a = ns->a, h.b = ns->b, h.c = ns->c, h.eps = ns->eps;
  return run(count, [&](int32_t i) {
    MuonTensor t = shape_of(m[i].rows, m[i].cols);
    t.in = m[i].in;
    t.out = m[i].out;
    t.ldi = (int32_t)m[i].ld_in;
    t.ldo = (int32_t)m[i].ld_out;
    t.bf16 = m[i].dtype == QLORA_BF16;
    return t;
  }, h, ws, ws_bytes, static_cast<hipStream_t>(stream));
}

qlora_status qlora_muon_step(const qlora_muon_hparams* p, const qlora_muon_tensor* tensors,
                             int32_t count, void* ws, size_t ws_bytes, void* stream) {
  if (!p || !valid_ns(&p->ns) || !(p->lr >= 0) || !std::isfinite(p->lr) ||
      !(p->momentum >= 0 && p->momentum < 1) || !(p->weight_decay >= 0) ||
      !std::isfinite(p->weight_decay) || (p->nesterov != 0 && p->nesterov != 1) ||
      p->adjust < QLORA_MUON_PLAIN || p->adjust > QLORA_MUON_RMS || count < 0 ||
      (count > 0 && !tensors))
    return QLORA_ERR_INVALID_ARG;
  for (int32_t i = 0; i < count; ++i) {
    const qlora_muon_tensor& t = tensors[i];
    if (!valid_type(t.grad_dtype) || t.reserved != 0) return QLORA_ERR_INVALID_ARG;
    const qlora_status st = check_shape(t.rows, t.cols);
    if (st != QLORA_OK) return st;
    if (t.rows == 0 || t.cols == 0) continue;
    if (!valid_matrix(t.param, 4, t.ld_param, t.cols) ||
        !valid_matrix(t.grad, esize(t.grad_dtype), t.ld_grad, t.cols) ||
        !valid_matrix(t.momentum, 4, t.ld_momentum, t.cols) ||
        (t.param_bf16 && !valid_matrix(t.param_bf16, 2, t.ld_bf16, t.cols)))
      return QLORA_ERR_INVALID_ARG;
  }
  MuonHyper h = {};
  h.mu = (float)p->momentum;
  h.one_minus_mu = (float)(1.0 - p->momentum);
  h.decay = (float)(1.0 - p->lr * p->weight_decay);
  h.nesterov = p->nesterov;
  h.step = 1;
  h.steps = p->ns.steps;
  h.a = p->ns.a, h.b = p->ns.b, h.c = p->ns.c, h.eps = p->ns.eps;
  return run(count, [&](int32_t i) {
    const qlora_muon_tensor& x = tensors[i];
    MuonTensor t = shape_of(x.rows, x.cols);
    t.in = x.grad;
    t.m = x.momentum;
    t.out = x.param;
    t.pb = x.param_bf16;
    t.ldi = (int32_t)x.ld_grad;
    t.ldm = (int32_t)x.ld_momentum;
    t.ldo = (int32_t)x.ld_param;
    t.ldb = (int32_t)x.ld_bf16;
    t.bf16 = x.grad_dtype == QLORA_BF16;
    const double rows = (double)x.rows, cols = (double)x.cols;
    const double f = p->adjust == QLORA_MUON_RMS     ? 0.2 * std::sqrt(rows > cols ? rows : cols)
                     : p->adjust == QLORA_MUON_SHAPE ? std::sqrt(rows > cols ? rows / cols : 1.0)
                                                     : 1.0;
    t.scale = (float)(p->lr * f);
    return t;
  }, h, ws, ws_bytes, static_cast<hipStream_t>(stream));
}

}  // extern "C"
