// Losses on packed logits: token log-probabilities, the preference loss over
// pairs and the clipped policy loss, with the gradient of the logits.  The
// logits are all of the work: a few bytes of loss per row of a vocabulary's
// length, so every kernel that reads them is a stream bound by HBM, and the
// arithmetic between the streams (float64, per row or sequence) is kept to
// one small launch.
//
//     logp = z_y - m - log s,   m = max z,   s = sum exp(z - m)
//     dz_v = w (1[v == y] - exp(z_v - m) / s),   w = dLoss / dlogp
#include <cmath>

#include "loss.h"
#include "skinny.h"

namespace qnf4 {
namespace {

constexpr int kT = 256;          // threads of a workgroup
constexpr int kBatch = 8;        // 16-byte loads a thread has in flight
constexpr float kInf = __builtin_inff();

// exp(d), d <= 0 or NaN; log2(e) as the nearest float32 and what that lacks
constexpr float kL2e = 0x1.715476p+0f, kL2eLow = 0x1.4ae0bep-26f;
__device__ __forceinline__ float exp_f32(float d) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(d, kL2eLow, d * kL2e));
}

// The same to within v_exp_f32's own error, whatever the argument's size: what
// the product d log2(e) was rounded by comes back as a factor.
__device__ __forceinline__ float exp_exact(float d) {
  const float t = d * kL2e, x = __builtin_amdgcn_exp2f(t);
  const float rest = __builtin_fmaf(d, kL2eLow, __builtin_fmaf(d, kL2e, -t));
  return d > -200.f ? __builtin_fmaf(x, 0.6931472f * rest, x) : x;
}

// A row's sum is taken over 2^(z H - R), H the 16 leading bits of log2(e) and R
// an integer near the maximum's: for a bf16 z that argument is exact wherever
// |z| is of the maximum's size, so the exponentials that make up the sum carry
// v_exp_f32's own error only (2.6e-8, mean -3e-9).  With the rounded argument
// of exp_f32 the few hundred values a bf16 takes there leave every row's sum
// 6e-8 too large, which a sequence's sum of log ratios adds up.  What H lacks
// is first order: 2^(z D) = 2^(m D) (1 + (z - m) D ln 2), from sum v z.
// x y with 0 times anything 0 (v_mul_legacy_f32): a masked logit's x is 0
__device__ float mul_zero(float x, float y) __asm("llvm.amdgcn.fmul.legacy");

constexpr float kH = 0x1.7154p+0f;
constexpr float kDLn2 = 0x1.480fb6p-18f;   // (log2(e) - kH) ln 2

template <typename T>
__device__ __forceinline__ float ld1(const T* p) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(*p);
  else return *p;
}
template <typename T>
__device__ __forceinline__ void st1(T* p, float v) {
  if constexpr (sizeof(T) == 2) *p = to_bf16(v);
  else *p = v;
}
template <typename T>
constexpr int vec() { return 16 / (int)sizeof(T); }   // values of a 16-byte chunk

template <typename T>
__device__ __forceinline__ void unpack(const uint4& q, float (&f)[vec<T>()]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      f[2 * i] = __builtin_bit_cast(float, w[i] << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
    } else {
      f[i] = __builtin_bit_cast(float, w[i]);
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[vec<T>()]) {
  if constexpr (sizeof(T) == 2)
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  else
    return __builtin_bit_cast(uint4, f32x4_t{f[0], f[1], f[2], f[3]});
}
// a chunk of -inf: what stands in for values past a row's end
template <typename T>
__device__ __forceinline__ uint4 no_values() {
  const uint32_t w = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
  return make_uint4(w, w, w, w);
}

// A row of any alignment: `head` values up to the first 16-byte boundary, `nb`
// whole chunks from there, and a tail; head and tail (at most 14 values) are
// the edge, one value to a thread.
template <typename T>
struct Row {
  const T* z;
  int head, edge;
  int64_t nb, vocab;
  __device__ __forceinline__ Row(const LogitsView& v, int64_t t) {
    z = static_cast<const T*>(v.z) + t * v.ld;
    vocab = v.vocab;
    const int64_t off = (int64_t)((uintptr_t)z & 15) / (int64_t)sizeof(T);
    const int64_t h = off ? vec<T>() - off : 0;
    head = (int)(h < vocab ? h : vocab);
    nb = (vocab - head) / vec<T>();
    edge = (int)(vocab - nb * vec<T>());
  }
  __device__ __forceinline__ const uint4* body() const {
    return reinterpret_cast<const uint4*>(z + head);
  }
  // value index of edge element k
  __device__ __forceinline__ int64_t edge_at(int k) const {
    return k < head ? k : nb * vec<T>() + k;
  }
};

// sequence bounds, clamped to the rows there are
__device__ __forceinline__ int64_t cu_at(const LogitsView& v, int i) {
  const int64_t c = v.cu[i];
  return c < 0 ? 0 : c > v.rows ? v.rows : c;
}
__device__ __forceinline__ bool outside(const LogitsView& v, int64_t t) {
  return v.cu && (t < cu_at(v, 0) || t >= cu_at(v, v.nseq));
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) x = fmaxf(x, __shfl_xor(x, k));
  return x;
}
template <typename F>
__device__ __forceinline__ F wave_sum(F x) {
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) x += __shfl_xor(x, k);
  return x;
}

// Joins the threads' parts of a row in a fixed order; the result in every
// thread.  red: 2 floats for each wave.
template <int W>
__device__ __forceinline__ MaxSum wg_join(MaxSum a, float (*red)[2]) {
  const int wv = threadIdx.x >> 6;
  float m = wave_max(a.m);
  if ((threadIdx.x & 63) == 0) red[wv][0] = m;
  __syncthreads();
  m = red[0][0];
#pragma unroll
  for (int w = 1; w < W; ++w) m = fmaxf(m, red[w][0]);
  // a thread without values has m = -inf and s = 0 (or NaN, which stays)
  const float s = wave_sum(a.m == m ? a.s : a.s * exp_exact(a.m - m));
  if ((threadIdx.x & 63) == 0) red[wv][1] = s;
  __syncthreads();
  float t = red[0][1];
#pragma unroll
  for (int w = 1; w < W; ++w) t += red[w][1];
  return MaxSum{m, t};
}

// Adds a batch of chunks to a thread's part: the maximum first, so that the
// sum is rescaled once a batch.
template <typename T, int N>
__device__ __forceinline__ void add_batch(MaxSum& a, const uint4 (&q)[N]) {
  float m = a.m;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float f[vec<T>()];
    unpack<T>(q[i], f);
#pragma unroll
    for (int e = 0; e < vec<T>(); ++e) m = fmaxf(m, f[e]);
  }
  if (m > a.m) {
    a.s *= exp_exact(a.m - m);
    a.m = m;
  }
  if (__builtin_fabsf(m) < 0x1p20f) {
    const float R = __builtin_rintf(m * kH);
    float s = 0.f, sz = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float f[vec<T>()];
      unpack<T>(q[i], f);
#pragma unroll
      for (int e = 0; e < vec<T>(); ++e) {
        const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(f[e], kH, -R));
        s += x;
        sz += mul_zero(x, f[e]);
      }
    }
    // relative to the maximum itself: 2^(R - m H)
    a.s += __builtin_fmaf(kDLn2, __builtin_fmaf(-m, s, sz), s) *
           __builtin_amdgcn_exp2f(__builtin_fmaf(-m, kH, R));
  } else {   // no value yet, or of a size (or an infinity) the above cannot scale
    const float ref = m == -kInf ? 0.f : m;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float f[vec<T>()];
      unpack<T>(q[i], f);
#pragma unroll
      for (int e = 0; e < vec<T>(); ++e) a.s += exp_f32(f[e] - ref);
    }
  }
}
__device__ __forceinline__ void add_value(MaxSum& a, float x) {
  if (x > a.m) {
    a.s *= exp_exact(a.m - x);
    a.m = x;
  }
  a.s += exp_exact(x - (a.m == -kInf ? 0.f : a.m));
}

// ------------------------------------------------------------ row statistics
// Workgroup (row, slice of its chunks); 8 loads a thread in flight.  One slice
// writes the row's result, several their parts.
template <typename T>
__global__ __launch_bounds__(kT) void k_row_stats(LogitsView v, RowOut o, int slices) {
  __shared__ float red[kT / 64][2];
  if (blockIdx.x == 0 && threadIdx.x == 0 && o.ticket) *o.ticket = 0;
  const int64_t t = blockIdx.x / (unsigned)slices;
  const int sl = (int)(blockIdx.x - t * slices);
  if (t >= v.rows) return;
  const int64_t y = v.labels[t];
  if (y < 0 || y >= v.vocab || outside(v, t)) {
    if (sl == 0 && threadIdx.x == 0) {
      const float none = y < v.vocab || outside(v, t) ? 0.f : __builtin_nanf("");
      o.stats[t] = MaxSum{0.f, none};
      o.logp[t] = none;
    }
    return;
  }
  const Row<T> r(v, t);
  const int64_t per = ceil_div(r.nb, slices);
  const int64_t c0 = sl * per, c1 = c0 + per < r.nb ? c0 + per : r.nb;
  const uint4* b = r.body();
  MaxSum a{-kInf, 0.f};
  int64_t c = c0 + threadIdx.x;
  for (; c0 < c1 && c - threadIdx.x + kT * kBatch <= c1; c += kT * kBatch) {
    uint4 q[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) q[i] = b[c + kT * i];
    add_batch<T>(a, q);
  }
  if (c - threadIdx.x < c1) {
    uint4 q[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      q[i] = c + kT * i < c1 ? b[c + kT * i] : no_values<T>();
    add_batch<T>(a, q);
  }
  if (sl == 0 && (int)threadIdx.x < r.edge) add_value(a, ld1(r.z + r.edge_at(threadIdx.x)));
  a = wg_join<kT / 64>(a, red);
  if (threadIdx.x != 0) return;
  if (slices > 1) {
    o.part[t * slices + sl] = a;
  } else {
    o.stats[t] = a;
    o.logp[t] = (float)((double)ld1(r.z + y) - (double)a.m - std::log((double)a.s));
  }
}

// The statistics of row t, joined from its slices in their order if there are
// several (and then stored with logp).  Rows with a target only.
template <typename T>
__device__ __forceinline__ double row_logp(const LogitsView& v, const RowOut& o, int slices,
                                           int64_t t) {
  const int64_t y = v.labels[t];
  if (y >= v.vocab) return (double)__builtin_nanf("");   // written with the statistics
  MaxSum a;
  if (slices > 1) {
    const MaxSum* p = o.part + t * slices;
    float m = -kInf;
    for (int i = 0; i < slices; ++i) m = fmaxf(m, p[i].m);
    float s = 0.f;
    for (int i = 0; i < slices; ++i) s += p[i].m == m ? p[i].s : p[i].s * exp_exact(p[i].m - m);
    a = MaxSum{m, s};
    o.stats[t] = a;
  } else {
    a = o.stats[t];
  }
  const float zy = ld1(static_cast<const T*>(v.z) + t * v.ld + y);
  const double l = (double)zy - (double)a.m - std::log((double)a.s);
  if (slices > 1) o.logp[t] = (float)l;
  return l;
}

template <typename T>
__global__ __launch_bounds__(kT) void k_row_join(LogitsView v, RowOut o, int slices) {
  const int64_t t = (int64_t)blockIdx.x * kT + threadIdx.x;
  if (t < v.rows && v.labels[t] >= 0) row_logp<T>(v, o, slices, t);
}

// --------------------------------------------------------------- row gradient
// Workgroup (row, 256 x 8 chunks): loads, then the same chunks' stores.  Rows
// go from the last to the first: the statistics launch left the last ones in
// the Infinity Cache.  A row of weight 0 is written and not read.
template <typename T>
__global__ __launch_bounds__(kT) void k_row_grad(LogitsView v, const MaxSum* stats, const float* w,
                                                 const float* g, T* dz, int64_t ldd, int slices) {
  const int64_t tr = blockIdx.x / (unsigned)slices;
  const int sl = (int)(blockIdx.x - tr * slices);
  const int64_t t = v.rows - 1 - tr;
  const int64_t y = v.labels[t];
  const float c = y < 0 ? 0.f : w[t] * (g ? *g : 1.f);
  const Row<T> r(v, t);
  T* const d = dz + t * ldd;
  const bool even = (((uintptr_t)d ^ (uintptr_t)r.z) & 15) == 0;   // 16-byte stores fit
  const int64_t c0 = (int64_t)sl * kT * kBatch + threadIdx.x;
  const uint4* b = r.body();
  uint4* const db = reinterpret_cast<uint4*>(d + r.head);
  auto store = [&](int64_t k, const uint4& q) {
    if (even) {
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, q),
                                  reinterpret_cast<u32x4_t*>(db + k));
    } else {
      float f[vec<T>()];
      unpack<T>(q, f);
#pragma unroll
      for (int e = 0; e < vec<T>(); ++e) st1(d + r.head + k * vec<T>() + e, f[e]);
    }
  };
  const bool at_edge = sl == 0 && (int)threadIdx.x < r.edge;
  if (c == 0.f) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (c0 + kT * i < r.nb) store(c0 + kT * i, make_uint4(0u, 0u, 0u, 0u));
    if (at_edge) d[r.edge_at(threadIdx.x)] = 0;
    return;
  }
  uint4 q[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i)
    if (c0 + kT * i < r.nb) q[i] = b[c0 + kT * i];
  const MaxSum a = stats[t];
  const float k = -c / a.s;
  const int64_t yb = y - r.head;
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int64_t at = c0 + kT * i;
    if (at >= r.nb) continue;
    float f[vec<T>()];
    unpack<T>(q[i], f);
#pragma unroll
    for (int e = 0; e < vec<T>(); ++e) f[e] = k * exp_f32(f[e] - a.m);
    if ((uint64_t)(yb - at * vec<T>()) < (uint64_t)vec<T>()) {
#pragma unroll
      for (int e = 0; e < vec<T>(); ++e) f[e] += at * vec<T>() + e == yb ? c : 0.f;
    }
    store(at, pack<T>(f));
  }
  if (at_edge) {
    const int64_t at = r.edge_at(threadIdx.x);
    st1(d + at, k * exp_f32(ld1(r.z + at) - a.m) + (at == y ? c : 0.f));
  }
}

// ------------------------------------------------------- between the streams
// Sum over the workgroup in a fixed order, the result in every thread; red: a
// double for each wave.
__device__ __forceinline__ double wg_sum(double x, double* red) {
  x = wave_sum(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int w = 1; w < kT / 64; ++w) x += red[w];
  return x;
}

// Whether this workgroup is the last of n to come here.  What each wrote
// through thread 0 before is then visible to the last one's device_load.
__device__ __forceinline__ bool last_of(uint32_t* ticket, uint32_t n) {
  __shared__ uint32_t k;
  if (threadIdx.x == 0)
    k = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return k == n - 1;
}
__device__ __forceinline__ double device_load(const double* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void device_store(double* p, double v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// w of the rows in no sequence, shared out over the workgroups
__device__ __forceinline__ void zero_outside(const LogitsView& v, float* w) {
  const int64_t b = cu_at(v, 0), e = cu_at(v, v.nseq);
  const int64_t step = (int64_t)gridDim.x * kT, at = (int64_t)blockIdx.x * kT + threadIdx.x;
  for (int64_t t = at; t < b; t += step) w[t] = 0.f;
  for (int64_t t = e + at; t < v.rows; t += step) w[t] = 0.f;
}

// Workgroup per pair; the last one adds the pairs' losses in their order.
template <typename T>
__global__ __launch_bounds__(kT) void k_preference(LogitsView v, RowOut o, PreferenceArgs a,
                                                   int slices) {
  __shared__ double red[kT / 64];
  const int p = blockIdx.x;
  double lr[2], n[2];
  zero_outside(v, o.w);
  for (int i = 0; i < 2; ++i) {
    const int64_t b = cu_at(v, 2 * p + i), e = cu_at(v, 2 * p + i + 1);
    double lp = 0, rf = 0, cnt = 0;
    for (int64_t t = b + threadIdx.x; t < e; t += kT) {
      if (v.labels[t] < 0) continue;
      const double l = row_logp<T>(v, o, slices, t);
      lp += l;
      rf += l - (a.ref ? (double)a.ref[t] : 0.0);
      cnt += 1;
    }
    lp = wg_sum(lp, red);
    lr[i] = wg_sum(rf, red);
    n[i] = wg_sum(cnt, red);
    if (!a.length_mean || n[i] < 1) n[i] = 1;
    lr[i] /= n[i];
    if (threadIdx.x == 0) {
      if (a.seq_logp) a.seq_logp[2 * p + i] = (float)(lp / n[i]);
      if (a.rewards) a.rewards[2 * p + i] = (float)(a.beta * lr[i]);
    }
  }
  const double h = lr[0] - lr[1], x = a.beta * h;
  double loss, dh;
  if (a.kind == 0) {
    // log(1 + exp(-x)), log(1 + exp(x)) and both sigmoids without overflow
    const double ex = std::exp(-std::fabs(x)), u = std::log1p(ex);
    const double ln = u + (x < 0 ? -x : 0), lp = u + (x > 0 ? x : 0);
    const double sp = x >= 0 ? 1 / (1 + ex) : ex / (1 + ex);
    const double sn = x >= 0 ? ex / (1 + ex) : 1 / (1 + ex);
    loss = (1 - a.smooth) * ln + a.smooth * lp;
    dh = -a.beta * ((1 - a.smooth) * sn - a.smooth * sp);
    if (x != x) loss = dh = x;
  } else if (a.kind == 1) {
    loss = x < 1 ? 1 - x : (x != x ? x : 0.0);
    dh = x < 1 ? -a.beta : (x != x ? x : 0.0);
  } else {
    const double d = h - 1 / (2 * a.beta);
    loss = d * d;
    dh = 2 * d;
  }
  for (int i = 0; i < 2; ++i) {
    const int64_t b = cu_at(v, 2 * p + i), e = cu_at(v, 2 * p + i + 1);
    const float wt = (float)((i ? -dh : dh) / n[i] / a.pairs);
    for (int64_t t = b + threadIdx.x; t < e; t += kT) o.w[t] = v.labels[t] < 0 ? 0.f : wt;
  }
  if (threadIdx.x == 0) device_store(a.pair_loss + p, loss);
  if (!last_of(o.ticket, gridDim.x)) return;
  double tot = 0;
  for (int k = threadIdx.x; k < a.pairs; k += kT) tot += device_load(a.pair_loss + k);
  tot = wg_sum(tot, red);
  if (threadIdx.x == 0) *a.loss = (float)(tot / a.pairs);
}

__global__ __launch_bounds__(kT) void k_policy_count(LogitsView v, PolicyArgs a) {
  __shared__ double red[kT / 64];
  const int i = blockIdx.x;
  double n = 0;
  for (int64_t t = cu_at(v, i) + threadIdx.x; t < cu_at(v, i + 1); t += kT) n += v.labels[t] >= 0;
  n = wg_sum(n, red);
  if (threadIdx.x == 0) a.count[i] = (int)n;
}

// All targets, and the sequences that have any.
struct Totals {
  double targets, filled;
};
__device__ __forceinline__ Totals totals(const PolicyArgs& a, int nseq, double* red) {
  double n = 0, f = 0;
  for (int j = threadIdx.x; j < nseq; j += kT) {
    n += a.count[j];
    f += a.count[j] > 0;
  }
  n = wg_sum(n, red);
  return Totals{n, wg_sum(f, red)};
}
// weight of one target of sequence i in the mean
__device__ __forceinline__ double share_of(const PolicyArgs& a, const Totals& n, int i) {
  if (a.reduction == 0) return n.targets > 0 ? 1 / n.targets : 0;
  return a.count[i] > 0 ? 1 / (a.count[i] * n.filled) : 0;
}

struct Term {
  double loss, kl, clipped, dlogp;
};
__device__ __forceinline__ Term policy_term(const PolicyArgs& a, double l, double A, int64_t t) {
  const double r = a.old_logp ? std::exp(l - (double)a.old_logp[t]) : (l == l ? 1.0 : l);
  const double u = -A * r, c = -A * (r < a.lo ? a.lo : r > a.hi ? a.hi : r);
  const bool cut = c > u;
  Term x{cut ? c : u, 0.0, cut ? 1.0 : 0.0, cut ? 0.0 : u};
  if (a.ref) {
    const double d = (double)a.ref[t] - l, em = std::expm1(d);
    x.kl = em - d;
    x.loss += a.kl_coef * x.kl;
    x.dlogp -= a.kl_coef * em;
  }
  return x;
}

// Workgroup per sequence; the last one adds the sequences' sums in their order.
template <typename T>
__global__ __launch_bounds__(kT) void k_policy(LogitsView v, RowOut o, PolicyArgs a, int slices) {
  __shared__ double red[kT / 64];
  const int i = blockIdx.x;
  zero_outside(v, o.w);
  const Totals n = totals(a, v.nseq, red);
  const double share = share_of(a, n, i);
  double loss = 0, kl = 0, cut = 0;
  for (int64_t t = cu_at(v, i) + threadIdx.x; t < cu_at(v, i + 1); t += kT) {
    if (v.labels[t] < 0) {
      o.w[t] = 0.f;
      continue;
    }
    const double A = (double)(a.token_adv ? a.adv[t] : a.adv[i]);
    const Term x = policy_term(a, row_logp<T>(v, o, slices, t), A, t);
    loss += x.loss;
    kl += x.kl;
    cut += x.clipped;
    o.w[t] = (float)(share * x.dlogp);
  }
  loss = wg_sum(loss, red);
  kl = wg_sum(kl, red);
  cut = wg_sum(cut, red);
  if (threadIdx.x == 0) {
    device_store(a.sums + 3 * i, share * loss);
    device_store(a.sums + 3 * i + 1, share * kl);
    device_store(a.sums + 3 * i + 2, cut);
  }
  if (!last_of(o.ticket, gridDim.x)) return;
  double x[3] = {0, 0, 0};
  for (int j = threadIdx.x; j < v.nseq; j += kT)
    for (int k = 0; k < 3; ++k) x[k] += device_load(a.sums + 3 * j + k);
  for (int k = 0; k < 3; ++k) x[k] = wg_sum(x[k], red);
  if (threadIdx.x == 0) {
    a.out[0] = (float)x[0];
    a.out[1] = (float)x[1];
    a.out[2] = (float)(x[2] / (n.targets > 0 ? n.targets : 1));
  }
}

// 16-byte chunks of a row, at most (one that starts between boundaries has fewer)
int64_t row_chunks(int64_t vocab, int bf16) { return ceil_div(vocab, bf16 ? 8 : 4); }

hipError_t row_stats(const LogitsView& v, const RowOut& o, int slices, hipStream_t s) {
  const int64_t blocks = v.rows > 0 ? v.rows * slices : 1;   // one sets the counter
  return launch_kernel(v.bf16 ? k_row_stats<uint16_t> : k_row_stats<float>,
                       dim3((unsigned)blocks), dim3(kT), s, v, o, slices);
}

}  // namespace

// Enough workgroups to fill the chip where the rows alone do not, each with a
// batch of loads for every thread.
int row_slices(const LogitsView& v) {
  if (v.rows == 0) return 1;
  const int64_t chunks = row_chunks(v.vocab, v.bf16);
  int64_t n = ceil_div(1024, v.rows);
  const int64_t most = ceil_div(chunks, (int64_t)kT * kBatch / 2);
  if (n > most) n = most;
  return (int)(n < 1 ? 1 : n);
}

int64_t row_grad_slices(int64_t vocab, int bf16) {
  return ceil_div(row_chunks(vocab, bf16), (int64_t)kT * kBatch);
}

hipError_t launch_row_logp(const LogitsView& v, const RowOut& o, hipStream_t s) {
  const int slices = row_slices(v);
  hipError_t e = row_stats(v, o, slices, s);
  if (e == hipSuccess && slices > 1)
    e = launch_kernel(v.bf16 ? k_row_join<uint16_t> : k_row_join<float>,
                      dim3((unsigned)ceil_div(v.rows, kT)), dim3(kT), s, v, o, slices);
  return e;
}

hipError_t launch_row_grad(const LogitsView& v, const MaxSum* stats, const float* w,
                           const float* g, void* dz, int64_t ldd, hipStream_t s) {
  if (v.rows == 0) return hipSuccess;
  const int slices = (int)row_grad_slices(v.vocab, v.bf16);
  const dim3 grid((unsigned)(v.rows * slices));
  if (v.bf16)
    return launch_kernel(k_row_grad<uint16_t>, grid, dim3(kT), s, v, stats, w, g,
                         static_cast<uint16_t*>(dz), ldd, slices);
  return launch_kernel(k_row_grad<float>, grid, dim3(kT), s, v, stats, w, g,
                       static_cast<float*>(dz), ldd, slices);
}

hipError_t launch_preference(const LogitsView& v, const RowOut& o, const PreferenceArgs& a,
                             hipStream_t s) {
  const int slices = row_slices(v);
  const hipError_t e = row_stats(v, o, slices, s);
  if (e != hipSuccess) return e;
  return launch_kernel(v.bf16 ? k_preference<uint16_t> : k_preference<float>,
                       dim3((unsigned)a.pairs), dim3(kT), s, v, o, a, slices);
}

hipError_t launch_policy(const LogitsView& v, const RowOut& o, const PolicyArgs& a,
                         hipStream_t s) {
  const int slices = row_slices(v);
  hipError_t e = row_stats(v, o, slices, s);
  if (e == hipSuccess)
    e = launch_kernel(k_policy_count, dim3((unsigned)v.nseq), dim3(kT), s, v, a);
  if (e == hipSuccess)
    e = launch_kernel(v.bf16 ? k_policy<uint16_t> : k_policy<float>, dim3((unsigned)v.nseq),
                      dim3(kT), s, v, o, a, slices);
  return e;
}

}  // namespace qnf4
