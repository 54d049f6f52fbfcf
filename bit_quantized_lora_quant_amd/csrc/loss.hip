// Losses on packed logits: token log-probabilities, the preference loss over
// pairs and the clipped policy loss, with the gradient of the logits.
#include <cmath>

#include "loss.h"
#include "skinny.h"

namespace qnf4 {
namespace {

constexpr int kT = 256;
constexpr float kLog2e = 1.4426950408889634f;

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

__device__ __forceinline__ float exp2_f32(float x) { return __builtin_amdgcn_exp2f(x); }

// sequence bounds, clamped to the rows there are
__device__ __forceinline__ int64_t cu_at(const LogitsView& v, int i) {
  const int64_t c = v.cu[i];
  return c < 0 ? 0 : c > v.rows ? v.rows : c;
}
__device__ __forceinline__ bool has_target(const LogitsView& v, int64_t t) {
  if (v.labels[t] < 0) return false;
  return !v.cu || (t >= cu_at(v, 0) && t < cu_at(v, v.nseq));
}

// (maximum, sum of exp(z - maximum)) of two parts of a row
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -__builtin_inff()) return MaxSum{m, a.s + b.s};
  return MaxSum{m, a.s * exp2_f32((a.m - m) * kLog2e) + b.s * exp2_f32((b.m - m) * kLog2e)};
}

template <typename T>
__global__ __launch_bounds__(kT) void k_row_stats(LogitsView v, RowOut o) {
  __shared__ MaxSum red[kT];
  const int64_t t = blockIdx.x;
  const int64_t y = v.labels[t];
  if (!has_target(v, t) || y >= v.vocab) {
    if (threadIdx.x == 0) {
      const float bad = has_target(v, t) ? __builtin_nanf("") : 0.f;
      o.stats[2 * t] = 0.f;
      o.stats[2 * t + 1] = bad;
      o.logp[t] = bad;
    }
    return;
  }
  const T* z = static_cast<const T*>(v.z) + t * v.ld;
  MaxSum a{-__builtin_inff(), 0.f};
  for (int64_t e = threadIdx.x; e < v.vocab; e += kT) {
    const float x = ld1(z + e);
    if (x != x) a.s = x;                               // NaN: the row's sum is NaN
    else if (x != -__builtin_inff()) a = join(a, MaxSum{x, 1.f});
  }
  red[threadIdx.x] = a;
  __syncthreads();
  for (int k = kT / 2; k > 0; k >>= 1) {
    if ((int)threadIdx.x < k) red[threadIdx.x] = join(red[threadIdx.x], red[threadIdx.x + k]);
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    a = red[0];
    o.stats[2 * t] = a.m;
    o.stats[2 * t + 1] = a.s;
    o.logp[t] = (float)((double)ld1(z + y) - (double)a.m - std::log((double)a.s));
  }
}

template <typename T>
__global__ __launch_bounds__(kT) void k_row_grad(LogitsView v, const float* stats, const float* w,
                                                 const float* g, T* dz, int64_t ldd) {
  const int64_t t = blockIdx.x;
  const int64_t y = v.labels[t];
  const float c = has_target(v, t) ? w[t] * (g ? *g : 1.f) : 0.f;
  const T* z = static_cast<const T*>(v.z) + t * v.ld;
  T* d = dz + t * ldd;
  if (c == 0.f) {
    for (int64_t e = threadIdx.x; e < v.vocab; e += kT) d[e] = 0;
    return;
  }
  const float m = stats[2 * t], sum = stats[2 * t + 1];
  for (int64_t e = threadIdx.x; e < v.vocab; e += kT) {
    const float p = exp2_f32((ld1(z + e) - m) * kLog2e) / sum;
    st1(d + e, e == y ? c * (1.f - p) : -c * p);
  }
}

// sum over the workgroup, in a fixed order; the result in every thread
__device__ __forceinline__ double wg_sum(double x, double* red) {
  red[threadIdx.x] = x;
  __syncthreads();
  for (int k = kT / 2; k > 0; k >>= 1) {
    if ((int)threadIdx.x < k) red[threadIdx.x] += red[threadIdx.x + k];
    __syncthreads();
  }
  x = red[0];
  __syncthreads();
  return x;
}

template <typename T>
__device__ __forceinline__ double row_logp(const LogitsView& v, const float* stats, int64_t t) {
  const int64_t y = v.labels[t];
  const float sum = stats[2 * t + 1];
  if (y >= v.vocab) return (double)__builtin_nanf("");
  const float zy = ld1(static_cast<const T*>(v.z) + t * v.ld + y);
  return (double)zy - (double)stats[2 * t] - std::log((double)sum);
}

template <typename T>
__global__ __launch_bounds__(kT) void k_preference(LogitsView v, RowOut o, PreferenceArgs a) {
  __shared__ double red[kT];
  const int p = blockIdx.x;
  double lr[2], n[2];
  for (int i = 0; i < 2; ++i) {
    const int64_t b = cu_at(v, 2 * p + i), e = cu_at(v, 2 * p + i + 1);
    double lp = 0, rf = 0, cnt = 0;
    for (int64_t t = b + threadIdx.x; t < e; t += kT) {
      if (v.labels[t] < 0) continue;
      const double l = row_logp<T>(v, o.stats, t);
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
    // log(1 + exp(-x)) and log(1 + exp(x)) without overflow
    const double u = std::log1p(std::exp(-std::fabs(x)));
    const double ln = u + (x < 0 ? -x : 0), lp = u + (x > 0 ? x : 0);
    loss = (1 - a.smooth) * ln + a.smooth * lp;
    const double ex = std::exp(-std::fabs(x));
    const double sp = x >= 0 ? 1 / (1 + ex) : ex / (1 + ex);     // sigmoid(x)
    const double sn = x >= 0 ? ex / (1 + ex) : 1 / (1 + ex);     // sigmoid(-x)
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
  if (threadIdx.x == 0) a.pair_loss[p] = loss;
  for (int i = 0; i < 2; ++i) {
    const int64_t b = cu_at(v, 2 * p + i), e = cu_at(v, 2 * p + i + 1);
    const float wt = (float)((i ? -dh : dh) / n[i] / a.pairs);
    for (int64_t t = b + threadIdx.x; t < e; t += kT) o.w[t] = v.labels[t] < 0 ? 0.f : wt;
  }
}

// rows in no sequence
__global__ __launch_bounds__(kT) void k_outside(LogitsView v, RowOut o) {
  const int64_t t = (int64_t)blockIdx.x * kT + threadIdx.x;
  if (t < v.rows && (t < cu_at(v, 0) || t >= cu_at(v, v.nseq))) o.w[t] = 0.f;
}

__global__ __launch_bounds__(kT) void k_preference_mean(PreferenceArgs a) {
  __shared__ double red[kT];
  double x = 0;
  for (int p = threadIdx.x; p < a.pairs; p += kT) x += a.pair_loss[p];
  x = wg_sum(x, red);
  if (threadIdx.x == 0) *a.loss = (float)(x / a.pairs);
}

__global__ __launch_bounds__(kT) void k_policy_count(LogitsView v, PolicyArgs a) {
  __shared__ double red[kT];
  const int i = blockIdx.x;
  double n = 0;
  for (int64_t t = cu_at(v, i) + threadIdx.x; t < cu_at(v, i + 1); t += kT) n += v.labels[t] >= 0;
  n = wg_sum(n, red);
  if (threadIdx.x == 0) a.count[i] = (int)n;
}

template <typename T>
__global__ __launch_bounds__(kT) void k_policy(LogitsView v, RowOut o, PolicyArgs a) {
  __shared__ double red[kT];
  const int i = blockIdx.x;
  double tot = 0, filled = 0;
  for (int j = threadIdx.x; j < v.nseq; j += kT) {
    tot += a.count[j];
    filled += a.count[j] > 0;
  }
  tot = wg_sum(tot, red);
  filled = wg_sum(filled, red);
  const double share = a.reduction == 0 ? (tot > 0 ? 1 / tot : 0)
                                        : (a.count[i] > 0 ? 1 / (a.count[i] * filled) : 0);
  double loss = 0, kls = 0, hits = 0;
  for (int64_t t = cu_at(v, i) + threadIdx.x; t < cu_at(v, i + 1); t += kT) {
    if (v.labels[t] < 0) {
      o.w[t] = 0.f;
      continue;
    }
    const double l = row_logp<T>(v, o.stats, t);
    const double A = (double)(a.token_adv ? a.adv[t] : a.adv[i]);
    const double r = std::exp(l - (a.old_logp ? (double)a.old_logp[t] : l));
    const double u = -A * r, c = -A * (r < a.lo ? a.lo : r > a.hi ? a.hi : r);
    const bool cut = c > u;
    double term = cut ? c : u, dterm = cut ? 0.0 : u;
    if (a.ref) {
      const double d = (double)a.ref[t] - l, em = std::expm1(d), kl = em - d;
      term += a.kl_coef * kl;
      dterm -= a.kl_coef * em;
      kls += kl;
    }
    loss += term;
    hits += cut;
    o.w[t] = (float)(share * dterm);
  }
  loss = wg_sum(loss, red);
  kls = wg_sum(kls, red);
  hits = wg_sum(hits, red);
  if (threadIdx.x == 0) {
    a.sums[4 * i] = share * loss;
    a.sums[4 * i + 1] = share * kls;
    a.sums[4 * i + 2] = hits;
    a.sums[4 * i + 3] = tot;
  }
}

__global__ __launch_bounds__(kT) void k_policy_sum(int nseq, PolicyArgs a) {
  __shared__ double red[kT];
  double x[3] = {0, 0, 0};
  for (int i = threadIdx.x; i < nseq; i += kT)
    for (int k = 0; k < 3; ++k) x[k] += a.sums[4 * i + k];
  for (int k = 0; k < 3; ++k) x[k] = wg_sum(x[k], red);
  if (threadIdx.x == 0) {
    a.out[0] = (float)x[0];
    a.out[1] = (float)x[1];
    a.out[2] = (float)(x[2] / fmax(a.sums[3], 1.0));
  }
}

}  // namespace

hipError_t launch_row_stats(const LogitsView& v, const RowOut& o, hipStream_t s) {
  if (v.rows == 0) return hipSuccess;
  return launch_kernel(v.bf16 ? k_row_stats<uint16_t> : k_row_stats<float>,
                       dim3((unsigned)v.rows), dim3(kT), s, v, o);
}

hipError_t launch_row_grad(const LogitsView& v, const float* stats, const float* w,
                           const float* g, void* dz, int64_t ldd, hipStream_t s) {
  if (v.rows == 0) return hipSuccess;
  if (v.bf16)
    return launch_kernel(k_row_grad<uint16_t>, dim3((unsigned)v.rows), dim3(kT), s, v, stats, w, g,
                         static_cast<uint16_t*>(dz), ldd);
  return launch_kernel(k_row_grad<float>, dim3((unsigned)v.rows), dim3(kT), s, v, stats, w, g,
                       static_cast<float*>(dz), ldd);
}

static hipError_t launch_outside(const LogitsView& v, const RowOut& o, hipStream_t s) {
  if (v.rows == 0) return hipSuccess;
  return launch_kernel(k_outside, dim3((unsigned)ceil_div(v.rows, kT)), dim3(kT), s, v, o);
}

hipError_t launch_preference(const LogitsView& v, const RowOut& o, const PreferenceArgs& a,
                             hipStream_t s) {
  hipError_t e = launch_row_stats(v, o, s);
  if (e == hipSuccess) e = launch_outside(v, o, s);
  if (e == hipSuccess)
    e = launch_kernel(v.bf16 ? k_preference<uint16_t> : k_preference<float>,
                      dim3((unsigned)a.pairs), dim3(kT), s, v, o, a);
  if (e == hipSuccess) e = launch_kernel(k_preference_mean, dim3(1), dim3(kT), s, a);
  return e;
}

hipError_t launch_policy(const LogitsView& v, const RowOut& o, const PolicyArgs& a,
                         hipStream_t s) {
  hipError_t e = launch_row_stats(v, o, s);
  if (e == hipSuccess) e = launch_outside(v, o, s);
  if (e == hipSuccess)
    e = launch_kernel(k_policy_count, dim3((unsigned)v.nseq), dim3(kT), s, v, a);
  if (e == hipSuccess)
    e = launch_kernel(v.bf16 ? k_policy<uint16_t> : k_policy<float>, dim3((unsigned)v.nseq),
                      dim3(kT), s, v, o, a);
  if (e == hipSuccess) e = launch_kernel(k_policy_sum, dim3(1), dim3(kT), s, v.nseq, a);
  return e;
}

}  // namespace qnf4
