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
// Bytes of the last rows that the statistics launch loads to stay cached (of the
// 256 MB Infinity Cache), for the gradient launch, which begins with them; the
// rows before go through without displacing them.  4096 x 128256, 3100 targets:
// statistics and gradient 131 + 314 us, 141 + 324 with plain loads, 125 + 337
// with none kept.
constexpr int64_t kKept = (int64_t)160 << 20;

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
// Keeps what was unpacked from a chunk from living on to its next use, and the
// chunks' work in order: 16 bytes of a row stay, not 8 floats.
__device__ __forceinline__ void forget(uint4& q) {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" : "+v"(q.x), "+v"(q.y), "+v"(q.z), "+v"(q.w));
}

// A row of any alignment: `head` values up to the first 16-byte boundary, `nb`
// whole chunks from there, and a tail; head and tail (at most 14 values) are
// the edge, one value to a thread.
template <typename T>
struct Row {
  const T* z;
  int head, edge, nb, vocab;
  __device__ __forceinline__ Row(const LogitsView& v, int64_t t) {
    z = static_cast<const T*>(v.z) + t * v.ld;
    vocab = (int)v.vocab;
    const int off = (int)((uintptr_t)z & 15) / (int)sizeof(T);
    const int h = off ? vec<T>() - off : 0;
    head = h < vocab ? h : vocab;
    nb = (vocab - head) / vec<T>();
    edge = vocab - nb * vec<T>();
  }
  // chunk k: a row is uniform in a workgroup, so its base stays in scalar
  // registers and a lane has a 32-bit offset
  __device__ __forceinline__ uint4 chunk(int k) const {
    return *reinterpret_cast<const uint4*>(at(k));
  }
  // the same, not to be kept by the caches
  __device__ __forceinline__ uint4 chunk_once(int k) const {
    return __builtin_bit_cast(
        uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(at(k))));
  }
  __device__ __forceinline__ const char* at(int k) const {
    return reinterpret_cast<const char*>(z + head) + (uint32_t)k * 16u;
  }
  // value index of edge element k
  __device__ __forceinline__ int edge_at(int k) const {
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
// thread, its sum also in float64 (`sum`): what is rounded once a thread comes
// out in the mean, what the last few additions round does not, and a sequence's
// log ratio or a KL term is small against its rows' logp.  S: float where
// the registers are short.
template <int W, typename S = double>
__device__ __forceinline__ MaxSum wg_join(MaxSum a, S (*red)[2], S* sum = nullptr) {
  const int wv = threadIdx.x >> 6;
  float m = wave_max(a.m);
  if ((threadIdx.x & 63) == 0) red[wv][0] = m;
  __syncthreads();
  m = (float)red[0][0];
#pragma unroll
  for (int w = 1; w < W; ++w) m = fmaxf(m, (float)red[w][0]);
  // a thread without values has m = -inf and s = 0 (or NaN, which stays)
  const S s = wave_sum((S)(a.m == m ? a.s : a.s * exp_exact(a.m - m)));
  if ((threadIdx.x & 63) == 0) red[wv][1] = s;
  __syncthreads();
  S t = red[0][1];
#pragma unroll
  for (int w = 1; w < W; ++w) t += red[w][1];
  if (sum) *sum = t;
  return MaxSum{m, (float)t};
}

// What turns a logit into its gradient: k exp(z - m), k = -w / sum.  A bf16
// gradient takes k into the exponent (one multiply-add; its argument is of the
// size of 20 at most where the value is not small, and its rounding then 2^-20,
// against a half bf16 step of 2^-8), a float32 one keeps the exponential apart.
// The target's is w (1 - p), formed as (w / sum) (sum - exp(z - m)): the
// difference is exact where p is next to 1 and what it leaves is small, so all of
// its error is the sum's own, where w - w p would bring p's rounding with it.
template <typename T>
struct GradOf {
  float m, s, ws, k;       // ws = w / sum
  uint32_t flip;           // bf16: k = log2 |ws|, flip: the sign of -w
  __device__ __forceinline__ GradOf(const MaxSum& a, float w) : m(a.m), s(a.s), ws(w / a.s), k(-ws) {
    flip = w > 0.f ? 0x80008000u : 0u;
    if constexpr (sizeof(T) == 2) k = __builtin_amdgcn_logf(__builtin_fabsf(ws));
  }
  // bf16: its magnitude
  __device__ __forceinline__ float value(float z) const {
    if constexpr (sizeof(T) == 2)
      return __builtin_amdgcn_exp2f(__builtin_fmaf(z - m, kL2e, k));
    else
      return k * exp_f32(z - m);
  }
  // the target's
  __device__ __forceinline__ float target(float z) const { return ws * (s - exp_exact(z - m)); }
  __device__ __forceinline__ float signed_value(float z) const {
    const float x = value(z);
    return sizeof(T) == 2 && flip ? -x : x;
  }
  // chunk `at` of a row whose target is body value yb; ty() its gradient
  template <typename F>
  __device__ __forceinline__ uint4 chunk(const uint4& q, int at, int yb, F ty) const {
    float f[vec<T>()];
    unpack<T>(q, f);
#pragma unroll
    for (int e = 0; e < vec<T>(); ++e) f[e] = value(f[e]);
    if ((unsigned)(yb - at * vec<T>()) < (unsigned)vec<T>()) {
      float t = ty();
      if (sizeof(T) == 2 && flip) t = -t;        // (flipped back below)
#pragma unroll
      for (int e = 0; e < vec<T>(); ++e) f[e] = at * vec<T>() + e == yb ? t : f[e];
    }
    uint4 o = pack<T>(f);
    if constexpr (sizeof(T) == 2) {
      o.x ^= flip; o.y ^= flip; o.z ^= flip; o.w ^= flip;
    }
    return o;
  }
};

// Adds a batch of chunks to a thread's part: the maximum first, so that the sum
// is rescaled once a batch.  Of a batch that is not FULL the first n chunks
// count and the others repeat one of them: that leaves the maximum alone, and a
// select keeps them out of the sums without a branch.
template <typename T, bool FULL, int N>
__device__ __forceinline__ void add_batch(MaxSum& a, uint4 (&q)[N], int n) {
  float m = a.m;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float f[vec<T>()];
    forget(q[i]);
    unpack<T>(q[i], f);
#pragma unroll
    for (int e = 0; e < vec<T>(); ++e) m = fmaxf(m, f[e]);
  }
  if (m > a.m) {
    a.s *= exp_exact(a.m - m);
    a.m = m;
  }
  const float R = __builtin_rintf(m * kH);
  float s = 0.f, sz = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float f[vec<T>()];
    forget(q[i]);
    unpack<T>(q[i], f);
    float c = 0.f, cz = 0.f;
#pragma unroll
    for (int e = 0; e < vec<T>(); ++e) {
      const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(f[e], kH, -R));
      c += x;
      cz = __builtin_fmaf(x, f[e], cz);
    }
    s += FULL || i < n ? c : 0.f;
    sz += FULL || i < n ? cz : 0.f;
  }
  // relative to the maximum itself: 2^(R - m H)
  s = __builtin_fmaf(kDLn2, __builtin_fmaf(-m, s, sz), s) *
      __builtin_amdgcn_exp2f(__builtin_fmaf(-m, kH, R));
  a.s += s;
}
// Whether a thread's part has to be summed again: a -inf (0 times it above), a
// NaN, or logits of a size H cannot scale.
__device__ __forceinline__ bool failed(const MaxSum& a) {
  return !(a.s < kInf) || (__builtin_fabsf(a.m) > 0x1p20f && a.m != -kInf);
}
// The sum of chunks c, c + step, .. below c1, against a maximum that is known.  A
// -inf sends its thread here: logp of 4096 x 128256 takes 189 us with the last 256
// columns masked by it and 283 with half of them (141 without, and with the type's
// lowest value in its place).
template <typename T>
__device__ __forceinline__ void sum_again(MaxSum& a, const Row<T>& r, int c, int c1, int step) {
  const float ref = a.m == -kInf ? 0.f : a.m;
  a.s = 0.f;
#pragma unroll 1
  for (; c < c1; c += step) {
    float f[vec<T>()];
    unpack<T>(r.chunk(c), f);
#pragma unroll
    for (int e = 0; e < vec<T>(); ++e) a.s += exp_exact(f[e] - ref);
  }
}
__device__ __forceinline__ void add_value(MaxSum& a, float x) {
  if (x > a.m) {
    a.s *= exp_exact(a.m - x);
    a.m = x;
  }
  a.s += exp_exact(x - (a.m == -kInf ? 0.f : a.m));
}

// Sums over the workgroup in a fixed order, the results in every thread; red: N
// doubles for each wave.
template <int NT, int N>
__device__ __forceinline__ void wg_sum(double (&x)[N], double (*red)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = wave_sum(x[i]);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[threadIdx.x >> 6][i] = x[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = red[0][i];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) x[i] += red[w][i];
  }
}

// The targets of sequence i, and its rows' sequence.
template <int NT>
__device__ __forceinline__ void count_sequence(const LogitsView& v, int i, int* count, int* seq,
                                               double (*red)[1]) {
  double n[1] = {0};
  for (int64_t t = cu_at(v, i) + threadIdx.x; t < cu_at(v, i + 1); t += NT) {
    n[0] += v.labels[t] >= 0;
    seq[t] = i;
  }
  wg_sum<NT, 1>(n, red);
  if (threadIdx.x == 0) count[i] = (int)n[0];
}

// ------------------------------------------------------------ row statistics
// Workgroup (row, slice of its chunks); 8 loads a thread in flight.  One slice
// writes the row's result, several their parts.  With `count` the first nseq
// workgroups count the sequences' targets instead.  Bound by HBM, with the
// exponentials close behind (9 operations a value, one of quarter rate): 0.80 GB
// of targets' rows in 131 us, 6.1 TB/s.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void k_row_stats(LogitsView v, RowOut o, int slices,
                                                  int* count, int* seq) {
  __shared__ double red[NT / 64][2];
  if (blockIdx.x == 0 && threadIdx.x == 0 && o.ticket) *o.ticket = 0;
  unsigned b = blockIdx.x;
  if (count) {
    if (b < (unsigned)v.nseq) {
      __shared__ double n[NT / 64][1];
      count_sequence<NT>(v, (int)b, count, seq, n);
      return;
    }
    b -= v.nseq;
  }
  const int64_t t = b / (unsigned)slices;
  const int sl = (int)(b - t * slices);
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
  const int per = (r.nb + slices - 1) / slices;
  const int c0 = sl * per < r.nb ? sl * per : r.nb, c1 = c0 + per < r.nb ? c0 + per : r.nb;
  MaxSum a{-kInf, 0.f};
  const int tid = threadIdx.x;
  int c = c0 + tid;
  const bool keep = (v.rows - t) * v.ld * (int64_t)sizeof(T) < kKept;
  for (; c - tid + NT * kBatch <= c1; c += NT * kBatch) {
    uint4 q[kBatch];
    if (keep) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) q[i] = r.chunk(c + NT * i);
    } else {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) q[i] = r.chunk_once(c + NT * i);
    }
    add_batch<T, true>(a, q, kBatch);
  }
  if (c < c1) {
    uint4 q[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      q[i] = r.chunk(c + NT * i < c1 ? c + NT * i : c);
    add_batch<T, false>(a, q, (c1 - c + NT - 1) / NT);
  }
  if (failed(a)) sum_again<T>(a, r, c0 + tid, c1, NT);
  if (sl == 0 && tid < r.edge) add_value(a, ld1(r.z + r.edge_at(tid)));
  double sum;
  a = wg_join<NT / 64>(a, red, &sum);
  if (threadIdx.x != 0) return;
  const float zy = ld1(r.z + y);
  if (sl == 0) o.zy[t] = zy;
  if (slices > 1) {
    o.part[t * slices + sl] = a;
  } else {
    o.stats[t] = a;
    o.logp[t] = (float)((double)zy - (double)a.m - std::log(sum));
  }
}

// The statistics of row t, joined from its slices in their order if there are
// several (and then stored with logp).  Rows with a target only.
__device__ __forceinline__ double row_logp(const LogitsView& v, const RowOut& o, int slices,
                                           int64_t t) {
  const int64_t y = v.labels[t];
  if (y >= v.vocab) return (double)__builtin_nanf("");   // written with the statistics
  MaxSum a;
  double s = 0;
  if (slices > 1) {
    const MaxSum* p = o.part + t * slices;
    // (a thread has this to itself: its loads go out 16 at a time)
    MaxSum q[16];
    auto load = [&](int i0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) q[i] = p[i0 + i < slices ? i0 + i : slices - 1];
    };
    float m = -kInf;
    for (int i0 = 0; i0 < slices; i0 += 16) {
      load(i0);
#pragma unroll
      for (int i = 0; i < 16; ++i) m = fmaxf(m, q[i].m);
    }
    for (int i0 = 0; i0 < slices; i0 += 16) {
      if (slices > 16) load(i0);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        s += i0 + i >= slices ? 0.f : q[i].m == m ? q[i].s : q[i].s * exp_exact(q[i].m - m);
    }
    a = MaxSum{m, (float)s};
    o.stats[t] = a;
  } else {
    a = o.stats[t];
    s = a.s;
  }
  const double l = (double)o.zy[t] - (double)a.m - std::log(s);
  if (slices != 1) o.logp[t] = (float)l;
  return l;
}

__global__ __launch_bounds__(kT) void k_row_join(LogitsView v, RowOut o, int slices) {
  const int64_t t = (int64_t)blockIdx.x * kT + threadIdx.x;
  if (t < v.rows && v.labels[t] >= 0) row_logp(v, o, slices, t);
}

// --------------------------------------------------------------- row gradient
// Workgroup (row, 256 x 8 chunks): loads, then the same chunks' stores.  Rows
// go from the last to the first: the statistics launch left the last ones in
// the Infinity Cache.  A row of weight 0 is written and not read.  Bound by HBM:
// 0.80 GB read and 1.05 GB written in 314 us, 5.9 TB/s.
template <typename T>
__global__ __launch_bounds__(kT) void k_row_grad(LogitsView v, const MaxSum* stats, const float* w,
                                                 const float* g, T* dz, int64_t ldd, int slices) {
  const int64_t tr = blockIdx.x / (unsigned)slices;
  const int sl = (int)(blockIdx.x - tr * slices);
  const int64_t t = v.rows - 1 - tr;
  const int64_t y = v.labels[t];
  const float wt = y < 0 ? 0.f : w[t];
  const float c = wt == 0.f ? 0.f : wt * (g ? *g : 1.f);   // (0 whatever g is)
  const Row<T> r(v, t);
  T* const d = dz + t * ldd;
  const bool even = (((uintptr_t)d ^ (uintptr_t)r.z) & 15) == 0;   // 16-byte stores fit
  const int c0 = sl * kT * kBatch + (int)threadIdx.x;
  char* const db = reinterpret_cast<char*>(d + r.head);
  auto store = [&](int k, const uint4& q) {
    if (even) {
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, q),
                                  reinterpret_cast<u32x4_t*>(db + (uint32_t)k * 16u));
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
    if (c0 + kT * i < r.nb) q[i] = r.chunk_once(c0 + kT * i);
  const GradOf<T> grad(stats[t], c);
  const int yb = y < v.vocab ? (int)y - r.head : -vec<T>();
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int at = c0 + kT * i;
    if (at >= r.nb) continue;
    forget(q[i]);
    store(at, grad.chunk(q[i], at, yb, [&] {   // (z_y is in this chunk; the row may be gone)
      float f[vec<T>()], zy = 0.f;
      unpack<T>(q[i], f);
#pragma unroll
      for (int e = 0; e < vec<T>(); ++e) zy = at * vec<T>() + e == yb ? f[e] : zy;
      return grad.target(zy);
    }));
  }
  if (at_edge) {
    const int at = r.edge_at(threadIdx.x);
    const float z = ld1(r.z + at);
    st1(d + at, at == y ? grad.target(z) : grad.signed_value(z));
  }
}

// ------------------------------------------------------- between the streams
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
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (int64_t t = at; t < b; t += step) w[t] = 0.f;
  for (int64_t t = e + at; t < v.rows; t += step) w[t] = 0.f;
}

// Workgroup per pair, its two sequences in one pass; the last one adds the
// pairs' losses in their order.
constexpr int kSeqT = 512;

__global__ __launch_bounds__(kSeqT) void k_preference(LogitsView v, RowOut o, PreferenceArgs a,
                                                      int slices) {
  __shared__ double red[kSeqT / 64][6];
  const int p = blockIdx.x;
  const int64_t b = cu_at(v, 2 * p), mid = cu_at(v, 2 * p + 1), e = cu_at(v, 2 * p + 2);
  double sum[6] = {0, 0, 0, 0, 0, 0};   // logp, log ratio, targets of either
  zero_outside(v, o.w);
  for (int64_t t = b + threadIdx.x; t < e; t += kSeqT) {
    if (v.labels[t] < 0) continue;
    const double l = row_logp(v, o, slices, t);
    const double d = l - (a.ref ? (double)a.ref[t] : 0.0);
    const bool second = t >= mid;
    sum[0] += second ? 0.0 : l;
    sum[1] += second ? 0.0 : d;
    sum[2] += second ? 0.0 : 1.0;
    sum[3] += second ? l : 0.0;
    sum[4] += second ? d : 0.0;
    sum[5] += second ? 1.0 : 0.0;
  }
  wg_sum<kSeqT, 6>(sum, red);
  double lr[2], n[2];
  for (int i = 0; i < 2; ++i) {
    n[i] = a.length_mean && sum[3 * i + 2] > 1 ? sum[3 * i + 2] : 1;
    lr[i] = sum[3 * i + 1] / n[i];
    if (threadIdx.x == 0) {
      if (a.seq_logp) a.seq_logp[2 * p + i] = (float)(sum[3 * i] / n[i]);
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
    // (without smoothing, a pair won by infinity has no loss)
    loss = (1 - a.smooth) * ln + (a.smooth > 0 ? a.smooth * lp : 0.0);
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
  const float w0 = (float)(dh / n[0] / a.pairs), w1 = (float)(-dh / n[1] / a.pairs);
  for (int64_t t = b + threadIdx.x; t < e; t += kSeqT)
    o.w[t] = v.labels[t] < 0 ? 0.f : t < mid ? w0 : w1;
  if (threadIdx.x == 0) device_store(a.pair_loss + p, loss);
  if (!last_of(o.ticket, gridDim.x)) return;
  __shared__ double last[kSeqT / 64][1];
  double tot[1] = {0};
  for (int k = threadIdx.x; k < a.pairs; k += kSeqT) tot[0] += device_load(a.pair_loss + k);
  wg_sum<kSeqT, 1>(tot, last);
  if (threadIdx.x == 0) *a.loss = (float)(tot[0] / a.pairs);
}

__device__ __forceinline__ void list_targets(const LogitsView& v, int* list) {
  __shared__ int count[2][kSeqT / 64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int n = 0;
  auto label = [&](int64_t t) { return t < v.rows ? v.labels[t] : -1; };
  int64_t y = label(threadIdx.x);
  for (int64_t t0 = 0, k = 0; t0 < v.rows; t0 += kSeqT, k ^= 1) {
    const int64_t t = t0 + threadIdx.x;
    const bool yes = y >= 0 && y < v.vocab && !outside(v, t);
    y = label(t + kSeqT);                       // the next rows', in flight
    const uint64_t in = __ballot(yes);
    if (lane == 0) count[k][wv] = __popcll(in);
    __syncthreads();
    int at = n + __popcll(in & ((1ull << lane) - 1));
    for (int w = 0; w < kSeqT / 64; ++w) {
      at += w < wv ? count[k][w] : 0;
      n += count[k][w];
    }
    if (yes) list[at] = (int)t;
  }
  if (threadIdx.x == 0) list[v.rows] = n;
}

// Before the one-pass form: a workgroup per sequence counts its targets, and one
// more lists all rows with a target, in order, to be shared out.
__global__ __launch_bounds__(kSeqT) void k_policy_count(LogitsView v, RowOut o, PolicyArgs a) {
  __shared__ double red[kSeqT / 64][1];
  const int i = blockIdx.x;
  if (i == 0 && threadIdx.x == 0) *o.ticket = 0;
  if (i == v.nseq) {
    list_targets(v, a.list);
    return;
  }
  count_sequence<kSeqT>(v, i, a.count, a.seq, red);
}

// All targets, and the sequences that have any.
struct Totals {
  double targets, filled;
};
template <int NT>
__device__ __forceinline__ Totals totals(const PolicyArgs& a, int nseq, double (*red)[2]) {
  double n[2] = {0, 0};
  for (int j = threadIdx.x; j < nseq; j += NT) {
    n[0] += a.count[j];
    n[1] += a.count[j] > 0;
  }
  wg_sum<NT, 2>(n, red);
  return Totals{n[0], n[1]};
}
// weight of one target of sequence i in the mean
__device__ __forceinline__ double share_of(const PolicyArgs& a, const Totals& n, int i) {
  if (a.reduction == 0) return n.targets > 0 ? 1 / n.targets : 0;
  return a.count[i] > 0 ? 1 / (a.count[i] * n.filled) : 0;
}

struct Term {
  double loss, kl, clipped, dlogp;
};
// The exponents of the ratio and of the KL term, logp = l.
struct Exponents {
  double ratio, kl;
};
__device__ __forceinline__ Exponents policy_exponents(const PolicyArgs& a, double l, int64_t t) {
  return Exponents{a.old_logp ? l - (double)a.old_logp[t] : (l == l ? 0.0 : l),
                   a.ref ? (double)a.ref[t] - l : 0.0};
}
// The term of a target, from its exponents x and r = exp(x.ratio), e = exp(x.kl).
// e - 1 is off by 2^-53, far less than e moves by with what logp is off by (3e-8),
// however small x.kl is.  An advantage or coefficient of 0 adds 0 to an infinite
// ratio or divergence too (a masked target has logp -inf).
__device__ __forceinline__ Term policy_term(const PolicyArgs& a, double A, const Exponents& x,
                                            double r, double e) {
  const double u = A == 0 && r == r ? 0.0 : -A * r;
  const double c = -A * (r < a.lo ? a.lo : r > a.hi ? a.hi : r);
  const bool cut = c > u;
  Term y{cut ? c : u, 0.0, cut ? 1.0 : 0.0, cut ? 0.0 : u};
  if (a.ref) {
    const double em = e - 1;
    y.kl = em < (double)kInf ? em - x.kl : em;   // (NaN stays)
    if (a.kl_coef > 0) {
      y.loss += a.kl_coef * y.kl;
      y.dlogp -= a.kl_coef * em;
    }
  }
  return y;
}

// Workgroup per sequence; the last one adds the sequences' sums in their order.
__global__ __launch_bounds__(kSeqT) void k_policy(LogitsView v, RowOut o, PolicyArgs a, int slices) {
  __shared__ double tred[kSeqT / 64][2], red[kSeqT / 64][3];
  const int i = blockIdx.x;
  zero_outside(v, o.w);
  const Totals n = totals<kSeqT>(a, v.nseq, tred);
  const double share = share_of(a, n, i);
  double sum[3] = {0, 0, 0};            // loss, kl, clipped
  for (int64_t t = cu_at(v, i) + threadIdx.x; t < cu_at(v, i + 1); t += kSeqT) {
    if (v.labels[t] < 0) {
      o.w[t] = 0.f;
      continue;
    }
    const double A = (double)(a.token_adv ? a.adv[t] : a.adv[i]);
    const Exponents d = policy_exponents(a, row_logp(v, o, slices, t), t);
    const Term x = policy_term(a, A, d, std::exp(d.ratio), std::exp(d.kl));
    sum[0] += x.loss;
    sum[1] += x.kl;
    sum[2] += x.clipped;
    o.w[t] = (float)(share * x.dlogp);
  }
  wg_sum<kSeqT, 3>(sum, red);
  if (threadIdx.x == 0) {
    device_store(a.sums + 3 * i, share * sum[0]);
    device_store(a.sums + 3 * i + 1, share * sum[1]);
    device_store(a.sums + 3 * i + 2, sum[2]);
  }
  if (!last_of(o.ticket, gridDim.x)) return;
  double x[3] = {0, 0, 0};
  for (int j = threadIdx.x; j < v.nseq; j += kSeqT)
    for (int k = 0; k < 3; ++k) x[k] += device_load(a.sums + 3 * j + k);
  wg_sum<kSeqT, 3>(x, red);
  if (threadIdx.x == 0) {
    a.out[0] = (float)x[0];
    a.out[1] = (float)x[1];
    a.out[2] = (float)(x[2] / (n.targets > 0 ? n.targets : 1));
  }
}

// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ float uniform(float x) {
  return __builtin_bit_cast(float, uniform(__builtin_bit_cast(int, x)));
}
__device__ __forceinline__ double uniform(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint64_t lo = (uint32_t)uniform((int)(uint32_t)b), hi = (uint32_t)uniform((int)(b >> 32));
  return __builtin_bit_cast(double, hi << 32 | lo);
}

// ------------------------------------------- policy loss in one pass
// The weight of a row hangs on that row's logp and on counts known from the
// labels, so a workgroup can hold its row in registers from the maximum to the
// gradient: the logits are read once where the statistics and the gradient as
// two launches read them twice.  A row of up to NT x NC chunks goes to NT
// threads, NC 16-byte chunks each (1024 x 16 holds 131,072 bf16 in half of a
// CU's registers).  The workgroups are persistent and the memory never waits
// for arithmetic: as a chunk's gradient is stored its registers take the same
// chunk of the workgroup's next row, and the sums run over four chunks at a
// time as they arrive.  1.85 GB in 379 us (4096 x 128256), 4.9 TB/s; as two
// launches 456.  logp, weight and loss are formed after, from the same
// statistics; here one wave forms the weight for the gradient, with the same
// float64 operations, so that both say of a ratio next to a border whether it is
// clipped.  What is the same in all lanes is kept in scalar registers: a row's
// float64 constants beside it would spill (22 registers), and with more than 128
// a CU would hold fewer workgroups (64,000 bf16 logits, 512 threads: 132 us
// instead of 115 at 2048 rows).
template <typename T, int NT, int NC>
__global__ __launch_bounds__(NT, 4) void k_policy_rows(LogitsView v, RowOut o, PolicyArgs a, T* dz,
                                                       int64_t ldd) {
  __shared__ float red[NT / 64][2], row_w;
  __shared__ double dred[NT / 64][2];
  constexpr int kSum = 4;                       // chunks summed at a time
  Totals n = totals<NT>(a, v.nseq, dred);
  n = Totals{uniform(n.targets), uniform(n.filled)};
  const int64_t step = gridDim.x;
  auto has_target = [&](int64_t t) {
    const int64_t y = v.labels[t];
    return y >= 0 && y < v.vocab && !outside(v, t);
  };
  // every step-th of the rows with a target: as many for each workgroup, to one
  const int rows_with = uniform(a.list[v.rows]);
  auto listed = [&](int64_t k) { return k < rows_with ? (int64_t)uniform(a.list[k]) : v.rows; };
  auto store = [&](T* d, int head, int k, const uint4& q) {
    __builtin_nontemporal_store(
        __builtin_bit_cast(u32x4_t, q),
        reinterpret_cast<u32x4_t*>(reinterpret_cast<char*>(d + head) + (uint32_t)k * 16u));
  };
  // the workgroup's rows without a target: zeros (NaN for a label out of range)
  for (int64_t t = blockIdx.x; t < v.rows; t += step) {
    if (has_target(t)) continue;
    const Row<T> r(v, t);
    T* const d = dz + t * ldd;
    const float none = v.labels[t] >= v.vocab && !outside(v, t) ? __builtin_nanf("") : 0.f;
    uint4 q;
    if constexpr (sizeof(T) == 2) q.x = pack_bf16x2(none, none);
    else q.x = __builtin_bit_cast(uint32_t, none);
    q.y = q.z = q.w = q.x;
    for (int k = threadIdx.x; k < r.nb; k += NT) store(d, r.head, k, q);
    if ((int)threadIdx.x < r.edge) st1(d + r.edge_at(threadIdx.x), none);
    if (threadIdx.x == 0) {
      o.stats[t] = MaxSum{0.f, none};
      o.logp[t] = none;
    }
  }
  int64_t k0 = blockIdx.x, t = listed(k0);
  if (t >= v.rows) return;
  uint4 q[NC];
  float ze, zy;
  auto load_edge = [&](const Row<T>& r, int64_t row, int tid) {
    ze = tid < r.edge ? ld1(r.z + r.edge_at(tid)) : -kInf;
    zy = ld1(r.z + v.labels[row]);
  };
  {
    const Row<T> r(v, t);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int k = (int)threadIdx.x + NT * i;
      q[i] = r.chunk_once(k < r.nb ? k : r.nb - 1);
    }
    load_edge(r, t, threadIdx.x);
  }
  while (t < v.rows) {
    // (opaque, or the chunks' offsets are kept in registers over the rows)
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    k0 += step;
    const int64_t tn = listed(k0);
    const Row<T> r(v, t), rn(v, tn < v.rows ? tn : t);
    const int nbn = tn < v.rows ? rn.nb : 1;    // (without a next row one chunk, unused)
    const int64_t y = uniform((int)v.labels[t]);
    const int sq = uniform(a.seq[t]);
    const double A = (double)uniform(a.token_adv ? a.adv[t] : a.adv[sq]);
    const double share = uniform(share_of(a, n, sq));
    // this thread's chunks; loads past a row's end repeat its last one
    const int mine = (r.nb - tid + NT - 1) / NT;
    MaxSum s{-kInf, 0.f};
#pragma unroll
    for (int i = 0; i < NC; i += kSum)
      add_batch<T, false>(s, *reinterpret_cast<uint4(*)[kSum]>(&q[i]), mine - i);
    if (mine <= 0) s = MaxSum{-kInf, 0.f};
    if (failed(s)) sum_again<T>(s, r, tid, r.nb, NT);
    if (tid < r.edge) add_value(s, ze);
    s = wg_join<NT / 64, float>(s, red);
    s = MaxSum{uniform(s.m), uniform(s.s)};
    if (tid == 0) {
      o.stats[t] = s;
      o.zy[t] = zy;
    }
    // the weight as k_policy forms it after this launch, from the same statistics;
    // two lanes of a wave take an exponential each
    if (tid < 64) {
      const Exponents x =
          policy_exponents(a, (double)zy - (double)s.m - std::log((double)s.s), t);
      const double e = std::exp(tid & 1 ? x.kl : x.ratio);
      const Term term = policy_term(a, A, x, __shfl(e, 0), __shfl(e, 1));
      if (tid == 0) row_w = (float)(share * term.dlogp);
    }
    __syncthreads();
    const float w = uniform(row_w);
    const GradOf<T> grad(s, w);
    const float ty = uniform(grad.target(zy));
    const int yb = (int)y - r.head;
    T* const d = dz + t * ldd;
    const float zt = ze;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int at = tid + NT * i;
      forget(q[i]);
      if (at < r.nb)
        store(d, r.head, at, w == 0.f ? make_uint4(0u, 0u, 0u, 0u)
                                      : grad.chunk(q[i], at, yb, [&] { return ty; }));
      q[i] = rn.chunk_once(at < nbn ? at : nbn - 1);
    }
    if (tid < r.edge) {
      const int at = r.edge_at(tid);
      st1(d + at, w == 0.f ? 0.f : at == y ? ty : grad.signed_value(zt));
    }
    if (tn < v.rows) load_edge(rn, tn, tid);
    t = tn;
  }
}

// 16-byte chunks of a row, at most (one that starts between boundaries has fewer)
int64_t row_chunks(int64_t vocab, int bf16) { return ceil_div(vocab, bf16 ? 8 : 4); }

hipError_t row_stats(const LogitsView& v, const RowOut& o, int slices, hipStream_t s,
                     int* count = nullptr, int* seq = nullptr) {
  // (one at least, which sets the counter)
  const int64_t blocks = (v.rows > 0 ? v.rows * slices : 1) + (count ? v.nseq : 0);
  return launch_kernel(v.bf16 ? k_row_stats<uint16_t, kT> : k_row_stats<float, kT>,
                       dim3((unsigned)blocks), dim3(kT), s, v, o, slices, count, seq);
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

// Rows that half fill the chip or fill it twice go whole to workgroups of 1024
// threads, not in slices that a second launch joins: 256 rows of 32000 bf16 in
// 8.0 us against 13.0, 512 in 12.2 against 13.4, 256 of 128256 in 15.3 against
// 20.1.  With 16 rows of 128256 a workgroup is too slow for a row (10.5 against
// 7.0); rows of less than two loads a thread (9000 bf16) lose as much as they
// gain, and so do the losses, whose own launch joins the slices.
static bool whole_rows(const LogitsView& v) {
  return v.rows >= 128 && v.rows <= 512 && row_chunks(v.vocab, v.bf16) >= 2048;
}

hipError_t launch_row_logp(const LogitsView& v, const RowOut& o, hipStream_t s) {
  if (whole_rows(v))
    return launch_kernel(v.bf16 ? k_row_stats<uint16_t, 1024> : k_row_stats<float, 1024>,
                         dim3((unsigned)v.rows), dim3(1024), s, v, o, 1, nullptr, nullptr);
  const int slices = row_slices(v);
  hipError_t e = row_stats(v, o, slices, s);
  if (e == hipSuccess && slices > 1)
    e = launch_kernel(k_row_join, dim3((unsigned)ceil_div(v.rows, kT)), dim3(kT), s, v, o, slices);
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
  return launch_kernel(k_preference, dim3((unsigned)a.pairs), dim3(kSeqT), s, v, o, a, slices);
}

template <typename T, int NT, int NC>
static hipError_t policy_rows(const LogitsView& v, const RowOut& o, const PolicyArgs& a, void* dz,
                              int64_t ldd, hipStream_t s) {
  const int64_t most = 256 * (1024 / NT);       // what the CUs hold at a time
  return launch_kernel(k_policy_rows<T, NT, NC>, dim3((unsigned)(v.rows < most ? v.rows : most)),
                       dim3(NT), s, v, o, a, static_cast<T*>(dz), ldd);
}

// threads that hold the row in 16 chunks each at most
template <typename T>
static hipError_t policy_rows_of(const LogitsView& v, const RowOut& o, const PolicyArgs& a,
                                 void* dz, int64_t ldd, hipStream_t s) {
  const int64_t chunks = row_chunks(v.vocab, v.bf16);
  if (chunks <= 256 * 16) return policy_rows<T, 256, 16>(v, o, a, dz, ldd, s);
  if (chunks <= 512 * 16) return policy_rows<T, 512, 16>(v, o, a, dz, ldd, s);
  return policy_rows<T, 1024, 16>(v, o, a, dz, ldd, s);
}
// The one-pass form where a row fits in registers and is long enough to be worth
// a workgroup (32 KB), the rows fill the chip, and the gradient's rows start
// where the logits' do between 16-byte boundaries.  Whole calls, one pass against
// two: over 128,256 bf16 logits 38 and 31 us at 128 rows, 43 and 46 at 256, 130
// and 125 at 1024, 220 and 240 at 2048, 398 and 460 at 4096; over 32,000 25 and 28
// at 256 rows, 66 and 69 at 2048; over 9,000 25 and 25 at 256, 40 and 36 at 2048.
static bool one_pass(const LogitsView& v, const void* dz, int64_t ldd) {
  const int64_t chunks = row_chunks(v.vocab, v.bf16);
  const uintptr_t apart =
      ((uintptr_t)dz - (uintptr_t)v.z) | (uintptr_t)((ldd - v.ld) * (v.bf16 ? 2 : 4));
  return chunks >= 2048 && chunks <= 1024 * 16 && v.rows >= 256 && (apart & 15) == 0;
}

hipError_t launch_policy(const LogitsView& v, const RowOut& o, const PolicyArgs& a, void* dz,
                         int64_t ldd, hipStream_t s) {
  const bool fused = dz && one_pass(v, dz, ldd);
  // (0 slices: the statistics are there, logp is not)
  const int slices = fused ? 0 : row_slices(v);
  hipError_t e;
  if (fused) {
    e = launch_kernel(k_policy_count, dim3((unsigned)v.nseq + 1), dim3(kSeqT), s, v, o, a);
    if (e == hipSuccess)
      e = v.bf16 ? policy_rows_of<uint16_t>(v, o, a, dz, ldd, s)
                 : policy_rows_of<float>(v, o, a, dz, ldd, s);
  } else {
    e = row_stats(v, o, slices, s, a.count, a.seq);
  }
  if (e == hipSuccess)
    e = launch_kernel(k_policy, dim3((unsigned)v.nseq), dim3(kSeqT), s, v, o, a, slices);
  if (e == hipSuccess && dz && !fused)
    e = launch_row_grad(v, o.stats, o.w, nullptr, dz, ldd, s);
  return e;
}

}  // namespace qnf4
