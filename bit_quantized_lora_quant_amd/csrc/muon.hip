// The adapters' orthogonalised update: momentum, then Newton-Schulz steps
//
//     X_0 = U / max(|U|_F, eps),  X_k+1 = a X_k + b (X_k X_k^T) X_k + c (X_k X_k^T)^2 X_k
//
// which move every singular value of U towards 1.  An adapter's short side is its
// rank s <= 128 and its long side n thousands, so the steps are not taken on X: each
// multiplies X by a polynomial of its own product matrix G_k = X_k X_k^T (s x s), and
// all of those commute, so with P_k = a + b G_k + c G_k^2
//
//     G_k+1 = P_k G_k P_k,  X_K = (P_K-1 ... P_0) X_0.
//
// U is read twice, once for G_0 and once to be multiplied by the whole polynomial
// Q = P_K-1 ... P_0, in place of three products of its size a step.
//
// G is kept in float64.  Q reaches a^K (485) where a singular value is small, and
// its slope there a^(3K-1) and more, so a G off by 2^-24 of its largest eigenvalue
// would move the small singular values of U by percents: forming G squares its
// condition, which the steps on X itself do not.  The products of two float32
// values are exact in float64, so G_0 is U's to 2^-53 per sum.
//
//   k_muon_gram   workgroup per slice of the long side: m <- mu m + (1 - mu) g, and its
//                 part of U U^T on v_mfma_f64_16x16x4 (upper triangle of tiles)
//   k_muon_poly   workgroup per tensor: the parts in order, |U|^2 as the trace, Q / |U|
//   k_muon_apply  workgroup per chunk of 4096 elements: O = Q U, then the parameter's
//                 update
//   k_muon_small  all three for a call of small matrices
//
// Bound: HBM for rank up to 32 (a step moves 30 bytes a parameter, 22 of them
// unavoidable: gradient and momentum are read again).  448 adapters of rank 16, 42
// million parameters: gram 101 us and apply 152 us, 5.0 TB/s both, where a large copy
// reaches 5.2; polynomials 14 us, ten launches of the table 27 us.  From a rank of 64
// the f64 matrix cores join in (70 TF: 2 s flops a value each for the product and Q U),
// and the polynomial of a few matrices, a chain of products on a CU each, weighs more:
// two 65B layers of rank 64 take 64 us for gram, 6 us for the sum, 31 us for the
// polynomial and 76 us for apply (strips of several chunks to a workgroup, loading the
// next chunk under a product, took 105: fewer waves in flight).
#include "muon.h"

#include <type_traits>

namespace qnf4 {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;        // groups of 4 neighbours per thread and chunk
constexpr int kBuf = 4096 + 4 * 128;   // floats of a chunk: sp rows of C + 4

typedef double f64x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f64x4_t mfma64(double a, double b, f64x4_t c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

// A tensor seen along its short side s (index i) and long side n (index l): element
// (i, l) lies at i ld + l of a wide matrix, l ld + i of a tall one.
struct View {
  bool tall;
  int s, n, sp, chunk;
};
__device__ __forceinline__ View view(const MuonTensor& t) {
  View v;
  v.tall = t.rows > t.cols;
  v.s = v.tall ? t.cols : t.rows;
  v.n = v.tall ? t.rows : t.cols;
  v.sp = muon_pad(v.s);
  v.chunk = muon_chunk(v.sp);
  return v;
}

__device__ __forceinline__ bool fits16(const void* p, int ld, int bytes) {
  return ((uintptr_t)p % (4 * bytes)) == 0 && ld % 4 == 0;
}

__device__ __forceinline__ void load4(float (&x)[4], const float* p, int valid, bool vec) {
  if (vec && valid == 4) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = e < valid ? p[e] : 0.f;
  }
}
__device__ __forceinline__ void load4(float (&x)[4], const uint16_t* p, int valid, bool vec) {
  if (vec && valid == 4) {
    const uint2 f = *reinterpret_cast<const uint2*>(p);
    x[0] = bf16_to_f32((uint16_t)f.x); x[1] = bf16_to_f32((uint16_t)(f.x >> 16));
    x[2] = bf16_to_f32((uint16_t)f.y); x[3] = bf16_to_f32((uint16_t)(f.y >> 16));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = e < valid ? bf16_to_f32(p[e]) : 0.f;
  }
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4], int valid, bool vec) {
  if (vec && valid == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < valid) p[e] = x[e];
  }
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&x)[4], int valid, bool vec) {
  const uint32_t lo = pack_bf16x2(x[0], x[1]), hi = pack_bf16x2(x[2], x[3]);
  if (vec && valid == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < valid) p[e] = (uint16_t)((e < 2 ? lo : hi) >> (16 * (e & 1)));
  }
}
__device__ __forceinline__ void load_in(float (&x)[4], const MuonTensor& t, int64_t off, int valid,
                                        bool vec) {
  if (t.bf16) load4(x, static_cast<const uint16_t*>(t.in) + off, valid, vec);
  else load4(x, static_cast<const float*>(t.in) + off, valid, vec);
}

// A thread's four units of a chunk, 4 neighbours in memory each: wide C / 4 of them a
// short index, tall 4 NT a long index (past the short side or the end they hold
// nothing).  In LDS element (i, l) of a chunk lies at i SI + l SL floats, with one of
// the strides 1.
template <int NT, bool TALL>
struct Chunk {
  static constexpr int C = 4096 / (16 * NT);
  int i0, l0, s, n;     // of unit 0; sides
  __device__ __forceinline__ Chunk(const View& v) : s(v.s), n(v.n) {
    const int tid = threadIdx.x % kThreads;
    i0 = TALL ? 4 * (tid % (4 * NT)) : tid / (C / 4);
    l0 = TALL ? tid / (4 * NT) : 4 * (tid % (C / 4));
  }
  __device__ __forceinline__ int i(int k) const { return TALL ? i0 : i0 + 4 * NT * k; }
  __device__ __forceinline__ int l(int k) const { return TALL ? l0 + 64 / NT * k : l0; }
  // how many of unit k's elements there are in the chunk that starts at `at`
  __device__ __forceinline__ int valid(int k, int at) const {
    const int left = TALL ? s - i0 : n - at - l0;
    const bool in = TALL ? at + l(k) < n : i(k) < s;
    return in ? (left < 0 ? 0 : left < 4 ? left : 4) : 0;
  }
  __device__ __forceinline__ int64_t off(int k, int at, int ld) const {
    return TALL ? (int64_t)(at + l(k)) * ld + i0 : (int64_t)i(k) * ld + at + l0;
  }
  template <int SI, int SL>
  __device__ __forceinline__ void put(float* u, int k, const float (&x)[4]) const {
    float* at = u + i(k) * SI + l(k) * SL;
    if constexpr ((TALL ? SI : SL) == 1) {
      *reinterpret_cast<float4*>(at) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) at[e * (TALL ? SI : SL)] = x[e];
    }
  }
  template <int SI, int SL>
  __device__ __forceinline__ void get(float (&x)[4], const float* u, int k) const {
    const float* at = u + i(k) * SI + l(k) * SL;
    if constexpr ((TALL ? SI : SL) == 1) {
      const float4 f = *reinterpret_cast<const float4*>(at);
      x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = at[e * (TALL ? SI : SL)];
    }
  }
};

__device__ __forceinline__ float momentum(float m, float g, const MuonHyper& h) {
  return h.mu * m + h.one_minus_mu * g;
}
// what is orthogonalised, from the new momentum
__device__ __forceinline__ float update(float m, float g, const MuonHyper& h) {
  return h.nesterov ? momentum(m, g, h) : m;
}

// ---------------------------------------------------------------------- gram
// Products of a chunk over this workgroup's waves.  Up to two tiles of rank (one or
// three products) a wave takes every fourth 4-long step and all of them; beyond, a
// wave takes every fourth product and all steps, which ones known to the compiler
// (a test of the wave in the loop costs as much as the products).
template <int NT>
struct Gram {
  static constexpr int kTiles = NT * (NT + 1) / 2;
  static constexpr bool kByStep = NT <= 2;
  static constexpr int kMine = kByStep ? kTiles : (kTiles + 3) / 4;
  static constexpr int C = 4096 / (16 * NT), pitch = C + 4;
  f64x4_t acc[kMine];
  __device__ __forceinline__ void init() {
#pragma unroll
    for (int k = 0; k < kMine; ++k) acc[k] = f64x4_t{0., 0., 0., 0.};
  }
  template <int WV>
  __device__ __forceinline__ void add_products(const float* at) {
#pragma unroll 2
    for (int l = 0; l < C; l += 4) {
      double x[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) x[i] = (double)at[i * 16 * pitch + l];
      int k = 0;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = i; j < NT; ++j, ++k)
          if ((k & 3) == WV) acc[k >> 2] = mfma64(x[i], x[j], acc[k >> 2]);
    }
  }
  __device__ __forceinline__ void add(const float* u, int lane, int wv) {
    const float* at = u + (lane & 15) * pitch + (lane >> 4);
    if constexpr (kByStep) {
#pragma unroll 4
      for (int l = 4 * wv; l < C; l += 16) {
        double x[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) x[i] = (double)at[i * 16 * pitch + l];
        int k = 0;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = i; j < NT; ++j, ++k) acc[k] = mfma64(x[i], x[j], acc[k]);
      }
    } else {
      switch (wv) {
        case 0: add_products<0>(at); break;
        case 1: add_products<1>(at); break;
        case 2: add_products<2>(at); break;
        default: add_products<3>(at); break;
      }
    }
  }
  // (buf: kTiles * 3 * 256 doubles where waves have parts of the same product)
  __device__ __forceinline__ void store(double* out, double* buf, int lane, int wv) {
    if (kByStep) {
      __syncthreads();
      if (wv > 0) {
#pragma unroll
        for (int k = 0; k < kMine; ++k)
          reinterpret_cast<f64x4_t*>(buf)[((wv - 1) * kMine + k) * 64 + lane] = acc[k];
      }
      __syncthreads();
      if (wv > 0) return;
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        f64x4_t v = acc[k];
#pragma unroll
        for (int w = 0; w < 3; ++w) v += reinterpret_cast<f64x4_t*>(buf)[(w * kMine + k) * 64 + lane];
        reinterpret_cast<f64x4_t*>(out)[k * 64 + lane] = v;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kMine; ++k)
        if (4 * k + wv < kTiles) reinterpret_cast<f64x4_t*>(out)[(4 * k + wv) * 64 + lane] = acc[k];
    }
  }
};

template <int NT, bool TALL>
__device__ __forceinline__ void gram(const MuonTensor& t, const View& v, const MuonHyper& h,
                                     int slice, double* out, float* u, double* buf) {
  // (of ten products two waves have three: not the same two in neighbouring workgroups)
  const int lane = threadIdx.x & 63;
  const int wv = (__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + 2 * (slice & 1)) & 3;
  const int first = slice * t.slice, end = first + t.slice < v.n ? first + t.slice : v.n;
  const bool vi = fits16(t.in, t.ldi, t.bf16 ? 2 : 4), vm = fits16(t.m, t.ldm, 4);
  const Chunk<NT, TALL> c(v);
  float g[kUnits][4], m[kUnits][4];
  auto load = [&](int at) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int valid = c.valid(k, at);
      load_in(g[k], t, c.off(k, at, t.ldi), valid, vi);
      if (t.m) load4(m[k], t.m + c.off(k, at, t.ldm), valid, vm);
    }
  };
  auto process = [&](int at, float* to) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      if (t.m) {
#pragma unroll
        for (int e = 0; e < 4; ++e) m[k][e] = momentum(m[k][e], g[k][e], h);
        store4(t.m + c.off(k, at, t.ldm), m[k], c.valid(k, at), vm);
#pragma unroll
        for (int e = 0; e < 4; ++e) g[k][e] = update(m[k][e], g[k][e], h);
      }
      c.template put<Gram<NT>::pitch, 1>(to, k, g[k]);
    }
  };
  Gram<NT> G;
  G.init();
  load(first);
  process(first, u);
  __syncthreads();
  // a chunk's loads fly under the products of the one before, and no barrier stands
  // between these and its momentum, so that waves are in different phases
  int cur = 0;
  for (int at = first; at < end; at += v.chunk) {
    const bool more = at + v.chunk < end;
    if (more) load(at + v.chunk);
    G.add(u + cur, lane, wv);
    if (more) {
      cur = kBuf - cur;
      process(at + v.chunk, u + cur);
    }
    __syncthreads();
  }
  G.store(out, buf, lane, wv);
}

// Fills the call's table from a batch of it: which tensor each slice and chunk is of.
__device__ __forceinline__ void note(const MuonTensor& t, const View& v, int index, int c0, int c1,
                                     const MuonScratch& s) {
  const int per = t.slice / v.chunk;
  for (int c = c0 + threadIdx.x; c < c1; c += kThreads) {
    s.owner[t.chunk + c] = index;
    if (c % per == 0) s.owner_wg[t.wg + c / per] = index;
  }
  if (threadIdx.x == 0 && c0 == 0) s.t[index] = t;
}
__global__ __launch_bounds__(kThreads) void k_muon_table(const MuonBatch bt, MuonScratch s) {
  const MuonTensor t = bt.t[blockIdx.x];
  const View v = view(t);
  note(t, v, bt.first + blockIdx.x, 0, (int)ceil_div(v.n, v.chunk), s);
}

// TABLE: the call's tensors are in the scratch, all of them in one launch; else
// they are this batch's, the call's only one, and go to the scratch from here.
// (A launch per padded rank that there is: workgroups of another return.)
template <int NT, bool TABLE>
__global__ __launch_bounds__(kThreads, NT <= 2 ? 5 : NT == 4 ? 4 : 2)
void k_muon_gram(const std::conditional_t<TABLE, int, MuonBatch> bt, MuonHyper h, MuonScratch s) {
  // (slices of a rank up to 32 are a single chunk)
  __shared__ __attribute__((aligned(16))) float u[NT <= 2 ? kBuf : 2 * kBuf];
  __shared__ __attribute__((aligned(32))) double buf[NT <= 2 ? 3 * Gram<NT>::kTiles * 256 : 1];
  const int lane = threadIdx.x & 63, wg = blockIdx.x;
  MuonTensor t;
  int i = 0;
  if constexpr (TABLE) {
    t = s.t[__builtin_amdgcn_readfirstlane(s.owner_wg[wg])];
  } else {
    const uint64_t before =
        __builtin_amdgcn_ballot_w64(lane < bt.count && bt.t[lane < bt.count ? lane : 0].wg <= wg);
    i = __builtin_amdgcn_readfirstlane(__popcll(before)) - 1;
    t = bt.t[i];
  }
  const View v = view(t);
  if (v.sp != 16 * NT) return;
  const int slice = wg - t.wg;
  if constexpr (!TABLE) {
    const int per = t.slice / v.chunk, all = (int)ceil_div(v.n, v.chunk);
    note(t, v, i, slice * per, (slice + 1) * per < all ? (slice + 1) * per : all, s);
  }
  double* out = s.part + ((size_t)t.part + (size_t)slice * Gram<NT>::kTiles) * 256;
  if (v.tall) gram<NT, true>(t, v, h, slice, out, u, buf);
  else gram<NT, false>(t, v, h, slice, out, u, buf);
}

// ----------------------------------------------------------------------- sum
// From a rank of 33 on the slices' parts are megabytes, more than k_muon_poly's one
// workgroup per tensor should read: a workgroup per tile and tensor adds them into
// the first slice's place (64 x 22016: 2 us in place of 15).
template <int NT>
__global__ __launch_bounds__(kThreads) void k_muon_sum(MuonScratch s) {
  __shared__ __attribute__((aligned(32))) f64x4_t buf[3 * 64];
  const MuonTensor t = s.t[blockIdx.y];
  const View v = view(t);
  if (v.sp != 16 * NT) return;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int slices = (int)ceil_div(v.n, t.slice);
  f64x4_t* at = reinterpret_cast<f64x4_t*>(s.part + ((size_t)t.part + blockIdx.x) * 256) + lane;
  f64x4_t g = f64x4_t{0., 0., 0., 0.};
#pragma unroll 8
  for (int p = wv; p < slices; p += 4) g += at[(size_t)p * Gram<NT>::kTiles * 64];
  if (wv > 0) buf[(wv - 1) * 64 + lane] = g;
  __syncthreads();
  if (wv > 0) return;
#pragma unroll
  for (int w = 0; w < 3; ++w) g += buf[w * 64 + lane];
  *at = g;
}

// ---------------------------------------------------------------------- poly
// Wave J holds column panel J of each matrix as MFMA results: register v of tile I is
// row 16 I + 4 v + lane / 16, which is also the B operand of inner indices
// 16 I + 4 v ..: so a product needs only its left factor in LDS.
template <int NT>
struct Panel {
  f64x4_t t[NT];
};
template <int NT>
__device__ __forceinline__ Panel<NT> times(const double* x, const Panel<NT>& b, int lane) {
  constexpr int pitch = 16 * NT + 2;
  const double* at = x + (lane & 15) * pitch + (lane >> 4);
  Panel<NT> r;
#pragma unroll
  for (int i = 0; i < NT; ++i) r.t[i] = f64x4_t{0., 0., 0., 0.};
#pragma unroll
  for (int k = 0; k < NT; ++k)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
        r.t[i] = mfma64(at[16 * i * pitch + 16 * k + 4 * v], b.t[k][v], r.t[i]);
      // (reads of later steps drawn up here would spill: three matrices live)
      if (NT == 8) __builtin_amdgcn_sched_barrier(0);
    }
  return r;
}
template <int NT>
__device__ __forceinline__ void put_panel(double* x, const Panel<NT>& p, int lane, int pan,
                                          bool own) {
  constexpr int pitch = 16 * NT + 2;
  double* at = x + (lane >> 4) * pitch + 16 * pan + (lane & 15);
  __syncthreads();
  if (own) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) at[(16 * i + 4 * v) * pitch] = p.t[i][v];
  }
  __syncthreads();
}

// What U is multiplied by, from the trace of U U^T.  No square of a float32 value other
// than 0 is lost in float64, so a trace of 0 is a zero matrix, whose result is 0 under
// any eps (whose reciprocal need not be finite); else this is below 2^149.
__device__ __forceinline__ double inverse_norm(double trace, double eps) {
  // (fmax drops a NaN: then every product shows it)
  return trace == 0. ? 0. : 1. / fmax(sqrt(trace), eps);
}
// Q / |U|; of a zero matrix 0, also where Q, powers of a then, is not finite.
__device__ __forceinline__ double scaled(double q, double inv, double trace) {
  return trace == 0. ? 0. : q * inv;
}

constexpr int poly_waves(int nt) { return nt < 4 ? 4 : nt; }
template <int NT>
struct PolyLds {
  static constexpr int pitch = 16 * NT + 2;
  __attribute__((aligned(16))) double x[16 * NT * pitch];
  __attribute__((aligned(32))) f64x4_t buf[NT < 4 ? 4 * Gram<NT>::kTiles * 64 : 1];
};
// Barriers of polynomial(): after the matrix, two of G, two of each P and of each next G.
__device__ __forceinline__ int poly_barriers(int steps) { return 1 + 2 + 2 * steps + 2 * (steps - 1); }
// Q / |U| of the product matrix whose upper triangle is (NT < 4) the sum over the
// waves of l.buf, else at `from`: to `out`, as k_muon_apply's left operands.
template <int NT>
__device__ __forceinline__ void polynomial(const MuonHyper& h, PolyLds<NT>& l, const f64x4_t* from,
                                           double* out, int lane, int wv) {
  constexpr int pitch = PolyLds<NT>::pitch;
  double* x = l.x;
  const f64x4_t* buf = l.buf;
  // both halves of the matrix
  int k = 0;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = i; j < NT; ++j, ++k) {
      if (k % poly_waves(NT) != wv) continue;
      f64x4_t g;
      if constexpr (NT < 4) {
        g = buf[k * 64 + lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) g += buf[(w * Gram<NT>::kTiles + k) * 64 + lane];
      } else {
        g = from[k * 64];
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = 16 * i + 4 * v + (lane >> 4), c = 16 * j + (lane & 15);
        x[r * pitch + c] = g[v];
        x[c * pitch + r] = g[v];
      }
    }
  __syncthreads();
  // (waves past the panels, there for the sum, repeat panel 0 and keep to the barriers)
  const bool own = wv < NT;
  const int pan = own ? wv : 0;
  double tr = 0;
  for (int r = lane; r < 16 * NT; r += 64) tr += x[r * (pitch + 1)];
#pragma unroll
  for (int d = 32; d; d >>= 1) tr += __shfl_xor(tr, d);
  const double inv = inverse_norm(tr, h.eps);
  Panel<NT> G, Q;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v)
      G.t[i][v] = x[(16 * i + 4 * v + (lane >> 4)) * pitch + 16 * pan + (lane & 15)] * inv * inv;
  put_panel<NT>(x, G, lane, pan, own);
  for (int n = 0; n < h.steps; ++n) {
    Panel<NT> P = times<NT>(x, G, lane);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        P.t[i][v] = h.b * G.t[i][v] + h.c * P.t[i][v];
        if (i == pan && 4 * v + (lane >> 4) == (lane & 15)) P.t[i][v] += h.a;
      }
    const bool last = n + 1 == h.steps;
    Panel<NT> U;
    if (!last) U = times<NT>(x, P, lane);          // G P
    put_panel<NT>(x, P, lane, pan, own);
    if (n == 0) Q = P;
    else Q = times<NT>(x, Q, lane);                // P Q
    if (!last) {
      G = times<NT>(x, U, lane);                   // P G P
      put_panel<NT>(x, G, lane, pan, own);
    }
  }
  // (Q symmetric) row tile `pan`, inner indices 16 i + 4 v .., a line a load
  if (!own) return;
  out += pan * 256 * NT + lane;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) out[(4 * i + v) * 64] = scaled(Q.t[i][v], inv, tr);
}

template <int NT>
__global__ __launch_bounds__(64 * poly_waves(NT)) void k_muon_poly(MuonHyper h, MuonScratch s) {
  __shared__ PolyLds<NT> l;
  const MuonTensor t = s.t[blockIdx.x];
  const View vw = view(t);
  if (vw.sp != 16 * NT) return;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const f64x4_t* from = reinterpret_cast<const f64x4_t*>(s.part + (size_t)t.part * 256) + lane;
  if constexpr (NT < 4) {
    // every fourth slice a wave, then the four in order
    const int slices = (int)ceil_div(vw.n, t.slice);
    f64x4_t g[Gram<NT>::kTiles];
#pragma unroll
    for (int k = 0; k < Gram<NT>::kTiles; ++k) g[k] = f64x4_t{0., 0., 0., 0.};
#pragma unroll 8
    for (int p = wv; p < slices; p += 4)
#pragma unroll
      for (int k = 0; k < Gram<NT>::kTiles; ++k)
        g[k] += from[((size_t)p * Gram<NT>::kTiles + k) * 64];
#pragma unroll
    for (int k = 0; k < Gram<NT>::kTiles; ++k) l.buf[(wv * Gram<NT>::kTiles + k) * 64 + lane] = g[k];
    __syncthreads();
  }
  polynomial<NT>(h, l, from, s.q + (size_t)t.q * 256, lane, wv);
}

// Rank 33 to 64: all matrices fit LDS, so a product is taken by its ten tiles on and above
// the diagonal alone and written to both sides, which also keeps every matrix exactly
// symmetric: operands are read along rows, 512 bytes a read.  Eight waves, two a SIMD
// (which has three, three, two and two tiles), so that one's reads, polynomial and
// stores run beside the other's products: 31 us (33 with four waves; 43 with whole
// matrices; the products of the fullest SIMD alone are 22).  G P and P Q in one loop,
// with their left factor read once, took 32.  (The waves meet at barriers in code of
// their own, the same number in each.)
constexpr int kSide = 64, kPitch = kSide + 2, kPoly64 = 512;
struct Tri {
  int i, j;
};
template <int WV>
struct Mine {
  static constexpr Tri all[8][2] = {{{0, 0}, {0, 1}}, {{1, 1}, {1, 2}}, {{2, 2}}, {{3, 3}},
                                    {{0, 2}},         {{1, 3}},         {{2, 3}}, {{0, 3}}};
  static constexpr Tri t[2] = {all[WV][0], all[WV][1]};
  static constexpr int n = WV < 2 ? 2 : 1;
};
template <int WV>
struct Tri3 {
  using M = Mine<WV>;
  f64x4_t c[M::n];
  // a b, both symmetric and commuting
  __device__ __forceinline__ void product(const double* a, const double* b, int lane) {
    const int at = (lane >> 4) * kPitch + (lane & 15);
#pragma unroll
    for (int k = 0; k < M::n; ++k) c[k] = f64x4_t{0., 0., 0., 0.};
#pragma unroll
    for (int s = 0; s < kSide; s += 4)
#pragma unroll
      for (int k = 0; k < M::n; ++k)
        c[k] = mfma64(a[at + s * kPitch + 16 * M::t[k].i], b[at + s * kPitch + 16 * M::t[k].j], c[k]);
  }
  __device__ __forceinline__ void put(double* x, int lane) const {
#pragma unroll
    for (int k = 0; k < M::n; ++k)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = 16 * M::t[k].i + 4 * v + (lane >> 4), q = 16 * M::t[k].j + (lane & 15);
        x[r * kPitch + q] = c[k][v];
        if (M::t[k].i != M::t[k].j) x[q * kPitch + r] = c[k][v];
      }
  }
  // a + b g + c times what it holds
  __device__ __forceinline__ void polynomial(const double* g, const MuonHyper& h, int lane) {
#pragma unroll
    for (int k = 0; k < M::n; ++k)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = 16 * M::t[k].i + 4 * v + (lane >> 4), q = 16 * M::t[k].j + (lane & 15);
        c[k][v] = h.b * g[r * kPitch + q] + h.c * c[k][v];
        if (r == q) c[k][v] += h.a;
      }
  }
};
template <int WV>
__device__ __forceinline__ void poly64(const MuonHyper& h, double* g, double* p, double* u,
                                       double* q, int lane) {
  Tri3<WV> x, y;
  for (int n = 0; n < h.steps; ++n) {
    const bool last = n + 1 == h.steps;
    x.product(g, g, lane);
    x.polynomial(g, h, lane);
    x.put(n == 0 ? q : p, lane);          // P; the first is Q as well
    __syncthreads();
    const double* pn = n == 0 ? q : p;
    if (!last) {
      x.product(pn, g, lane);
      x.put(u, lane);                     // G P
    }
    if (n > 0) {
      y.product(p, q, lane);
      __syncthreads();
      y.put(q, lane);                     // P Q
    }
    __syncthreads();
    if (!last) {
      x.product(pn, u, lane);
      // (with n == 0 only: the next step writes P elsewhere, so Q stays)
      x.put(g, lane);                     // P G P
      __syncthreads();
    }
  }
}
__global__ __launch_bounds__(kPoly64) void k_muon_poly64(MuonHyper h, MuonScratch s) {
  __shared__ __attribute__((aligned(16))) double x[4][kSide * kPitch];
  const MuonTensor t = s.t[blockIdx.x];
  if (view(t).sp != kSide) return;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  double* g = x[0];
  // (the slices' parts are summed by then)
  const f64x4_t* from = reinterpret_cast<const f64x4_t*>(s.part + (size_t)t.part * 256) + lane;
  int k = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = i; j < 4; ++j, ++k) {
      if ((k & 7) != wv) continue;
      const f64x4_t c = from[k * 64];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = 16 * i + 4 * v + (lane >> 4), q = 16 * j + (lane & 15);
        g[r * kPitch + q] = c[v];
        g[q * kPitch + r] = c[v];
      }
    }
  __syncthreads();
  double tr = g[lane * (kPitch + 1)];
#pragma unroll
  for (int d = 32; d; d >>= 1) tr += __shfl_xor(tr, d);
  const double inv = inverse_norm(tr, h.eps);
  __syncthreads();
  for (int e = threadIdx.x; e < kSide * kSide; e += kPoly64)
    g[(e >> 6) * kPitch + (e & 63)] *= inv * inv;
  __syncthreads();
  switch (wv) {
    case 0: poly64<0>(h, x[0], x[1], x[2], x[3], lane); break;
    case 1: poly64<1>(h, x[0], x[1], x[2], x[3], lane); break;
    case 2: poly64<2>(h, x[0], x[1], x[2], x[3], lane); break;
    case 3: poly64<3>(h, x[0], x[1], x[2], x[3], lane); break;
    case 4: poly64<4>(h, x[0], x[1], x[2], x[3], lane); break;
    case 5: poly64<5>(h, x[0], x[1], x[2], x[3], lane); break;
    case 6: poly64<6>(h, x[0], x[1], x[2], x[3], lane); break;
    default: poly64<7>(h, x[0], x[1], x[2], x[3], lane); break;
  }
  // as k_muon_apply's left operands, a line a load (Q symmetric: half its row tile wv / 2)
  double* out = s.q + (size_t)t.q * 256 + wv * 256 * 2 + lane;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    out[e * 64] = scaled(x[3][(4 * (8 * (wv & 1) + e) + (lane >> 4)) * kPitch + 16 * (wv >> 1) +
                              (lane & 15)], inv, tr);
}

// --------------------------------------------------------------------- apply
// U <- Q U of one chunk in LDS: wave w takes row tiles and columns of it.
template <int NT, int SI, int SL>
__device__ __forceinline__ void product(const double* q, float* u) {
  constexpr int C = 4096 / (16 * NT);
  constexpr int RW = NT < 4 ? NT : 4;         // waves along the short side
  constexpr int MI = NT / RW;                 // row tiles of a wave
  constexpr int CW = 4 / RW;                  // waves along the long side
  constexpr int MJ = C / 16 / CW;             // column tiles of a wave
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x % kThreads >> 6);
  const int wr = wv % RW, wc = wv / RW;
  f64x4_t o[MI][MJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < MJ; ++j) o[i][j] = f64x4_t{0., 0., 0., 0.};
  const float* at = u + (lane >> 4) * SI + (16 * wc * MJ + (lane & 15)) * SL;
  const double* aq = q + wr * MI * 256 * NT + lane;
#pragma unroll
  for (int k = 0; k < 4 * NT; ++k) {
    double a[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) a[i] = aq[i * 256 * NT + 64 * k];
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      const double x = (double)at[4 * k * SI + 16 * j * SL];
#pragma unroll
      for (int i = 0; i < MI; ++i) o[i][j] = mfma64(a[i], x, o[i][j]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < MJ; ++j)
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        u[(16 * (wr * MI + i) + 4 * r + (lane >> 4)) * SI +
          (16 * (wc * MJ + j) + (lane & 15)) * SL] = (float)o[i][j][r];
  __syncthreads();
}

// What becomes of a chunk of O in LDS; p: the parameters' values of a step.
template <int NT, bool TALL, int SI, int SL>
__device__ __forceinline__ void finish(const MuonTensor& t, const MuonHyper& h,
                                       const Chunk<NT, TALL>& c, int start, const float* u,
                                       const float (&p)[kUnits][4]) {
  const bool vo = fits16(t.out, t.ldo, !h.step && t.bf16 ? 2 : 4), vb = fits16(t.pb, t.ldb, 2);
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int valid = c.valid(k, start);
    const int64_t off = c.off(k, start, t.ldo);
    float x[4];
    c.template get<SI, SL>(x, u, k);
    if (!h.step) {
      if (t.bf16) store4(static_cast<uint16_t*>(t.out) + off, x, valid, vo);
      else store4(static_cast<float*>(t.out) + off, x, valid, vo);
      continue;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = p[k][e] * h.decay - t.scale * x[e];
    store4(static_cast<float*>(t.out) + off, x, valid, vo);
    if (t.pb) store4(t.pb + c.off(k, start, t.ldb), x, valid, vb);
  }
}

template <int NT, bool TALL>
__device__ __forceinline__ void load_param(float (&p)[kUnits][4], const MuonTensor& t,
                                           const Chunk<NT, TALL>& c, int start) {
  const bool vo = fits16(t.out, t.ldo, 4);
#pragma unroll
  for (int k = 0; k < kUnits; ++k)
    load4(p[k], static_cast<const float*>(t.out) + c.off(k, start, t.ldo), c.valid(k, start), vo);
}

// A chunk's place in LDS for the product alone: the four units' values of a thread side
// by side, and an operand (four short indices of 16 long ones) on 64 banks.
template <int NT, bool TALL>
struct ApplyLds {
  static constexpr int C = 4096 / (16 * NT);
  static constexpr int SI = TALL ? 1 : C + 16, SL = TALL ? 16 * NT + 4 : 1;
  static constexpr int kFloats = TALL ? C * SL : 16 * NT * SI;
};

// The chunk's loads are in flight before those of Q; several workgroups a CU hide one
// another's phases.
template <int NT, bool TALL>
__device__ __forceinline__ void apply(const MuonTensor& t, const View& v, const MuonHyper& h,
                                      int start, const double* q, float* u) {
  using A = ApplyLds<NT, TALL>;
  const bool vi = fits16(t.in, t.ldi, t.bf16 ? 2 : 4), vm = fits16(t.m, t.ldm, 4);
  const bool need_in = !t.m || h.nesterov;
  const Chunk<NT, TALL> c(v);
  float g[kUnits][4], m[kUnits][4], p[kUnits][4];
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int valid = c.valid(k, start);
    if (need_in) load_in(g[k], t, c.off(k, start, t.ldi), valid, vi);
    if (t.m) load4(m[k], t.m + c.off(k, start, t.ldm), valid, vm);
  }
  if (h.step) load_param(p, t, c, start);
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    if (t.m) {
#pragma unroll
      for (int e = 0; e < 4; ++e) g[k][e] = update(m[k][e], g[k][e], h);
    }
    c.template put<A::SI, A::SL>(u, k, g[k]);
  }
  __syncthreads();
  product<NT, A::SI, A::SL>(q, u);
  finish<NT, TALL, A::SI, A::SL>(t, h, c, start, u, p);
}

// Last chunks first: what the first launches read last is still in the Infinity
// Cache.
template <int NT>
__global__ __launch_bounds__(kThreads, 4) void k_muon_apply(MuonHyper h, MuonScratch s) {
  constexpr int kWide = ApplyLds<NT, false>::kFloats, kTall = ApplyLds<NT, true>::kFloats;
  __shared__ __attribute__((aligned(16))) float u[kWide > kTall ? kWide : kTall];
  const int c = gridDim.x - 1 - blockIdx.x;
  const MuonTensor t = s.t[__builtin_amdgcn_readfirstlane(s.owner[c])];
  const View v = view(t);
  if (v.sp != 16 * NT) return;
  const double* q = s.q + (size_t)t.q * 256;
  const int start = (c - t.chunk) * v.chunk;
  if (v.tall) apply<NT, true>(t, v, h, start, q, u);
  else apply<NT, false>(t, v, h, start, q, u);
}

// --------------------------------------------------------------------- small
// A call of small matrices: a workgroup takes one from its gradient to its update, in
// one launch, U and Q in LDS all the while, four waves a chunk: latency is all there is
// (8 x 1024 and 1024 x 8, a step 16.6 us in place of 20.2 with three launches; with four
// waves for all chunks 30).
template <int NT, bool TALL>
__device__ __forceinline__ void small(const MuonTensor& t, const View& v, const MuonHyper& h,
                                      float* u, PolyLds<NT>& l, double* q) {
  constexpr int kTiles = Gram<NT>::kTiles, SI = Gram<NT>::pitch;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3;
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
  const int at = group * Chunk<NT, TALL>::C;
  const bool vi = fits16(t.in, t.ldi, t.bf16 ? 2 : 4), vm = fits16(t.m, t.ldm, 4);
  const Chunk<NT, TALL> c(v);
  u += group * kBuf;
  float g[kUnits][4], m[kUnits][4], p[kUnits][4];
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int valid = c.valid(k, at);
    load_in(g[k], t, c.off(k, at, t.ldi), valid, vi);
    if (t.m) load4(m[k], t.m + c.off(k, at, t.ldm), valid, vm);
  }
  if (h.step) load_param(p, t, c, at);
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    if (t.m) {
#pragma unroll
      for (int e = 0; e < 4; ++e) m[k][e] = momentum(m[k][e], g[k][e], h);
      store4(t.m + c.off(k, at, t.ldm), m[k], c.valid(k, at), vm);
#pragma unroll
      for (int e = 0; e < 4; ++e) g[k][e] = update(m[k][e], g[k][e], h);
    }
    c.template put<SI, 1>(u, k, g[k]);
  }
  __syncthreads();
  Gram<NT> G;
  G.init();
  G.add(u, lane, wv);
  // the chunks' products, from the last on
  f64x4_t* buf = l.buf + wv * kTiles * 64 + lane;
  for (int from = kMuonSmall - 1; from >= 0; --from) {
    if (group == from) {
#pragma unroll
      for (int k = 0; k < kTiles; ++k) buf[k * 64] = G.acc[k];
    }
    __syncthreads();
    if (group == from - 1) {
#pragma unroll
      for (int k = 0; k < kTiles; ++k) G.acc[k] += buf[k * 64];
    }
    __syncthreads();
  }
  if (group == 0) {
    polynomial<NT>(h, l, nullptr, q, lane, wv);
  } else {
    // (the barriers of the waves that do)
    for (int k = 0; k < poly_barriers(h.steps); ++k) __syncthreads();
  }
  __syncthreads();
  product<NT, SI, 1>(q, u);
  finish<NT, TALL, SI, 1>(t, h, c, at, u, p);
}
template <int NT>
__global__ __launch_bounds__(kMuonSmall * kThreads) void k_muon_small(const MuonBatch bt,
                                                                      MuonHyper h) {
  __shared__ __attribute__((aligned(16))) float u[kMuonSmall * kBuf];
  __shared__ PolyLds<NT> l;
  __shared__ __attribute__((aligned(16))) double q[256 * NT * NT];
  const MuonTensor t = bt.t[blockIdx.x];
  const View v = view(t);
  if (v.sp != 16 * NT) return;
  if (v.tall) small<NT, true>(t, v, h, u, l, q);
  else small<NT, false>(t, v, h, u, l, q);
}

}  // namespace

int muon_slice(int sp, int64_t total) {
  // A rank of 16 leaves 2 KB of parts a slice (a chunk moves 48 KB), one of 64 20 KB and
  // of 128 72 KB: there as many chunks as leave 960 workgroups, about what runs at once
  // (two 65B layers of rank 64: 176 us for the whole step, with 1536 of them 187).
  const int64_t most = sp <= 32 ? 1 : sp == 64 ? 8 : 16;
  int64_t chunks = ceil_div(total, 960 * 4096);
  chunks = chunks < 1 ? 1 : chunks > most ? most : chunks;
  return (int)chunks * muon_chunk(sp);
}

hipError_t launch_muon_table(const MuonBatch& b, const MuonScratch& s, hipStream_t st) {
  return launch_kernel(k_muon_table, dim3((unsigned)b.count), dim3(kThreads), st, b, s);
}

template <int NT>
hipError_t launch_gram(const MuonBatch* b, dim3 grid, const MuonHyper& h, const MuonScratch& s,
                       hipStream_t st) {
  return b ? launch_kernel(k_muon_gram<NT, false>, grid, dim3(kThreads), st, *b, h, s)
           : launch_kernel(k_muon_gram<NT, true>, grid, dim3(kThreads), st, 0, h, s);
}
hipError_t launch_muon_gram(const MuonBatch* b, int sp, int wgs, const MuonHyper& h,
                            const MuonScratch& s, hipStream_t st) {
  const dim3 grid((unsigned)wgs);
  switch (sp) {
    case 16: return launch_gram<1>(b, grid, h, s, st);
    case 32: return launch_gram<2>(b, grid, h, s, st);
    case 64: return launch_gram<4>(b, grid, h, s, st);
    default: return launch_gram<8>(b, grid, h, s, st);
  }
}

hipError_t launch_muon_small(const MuonBatch& b, int sp, const MuonHyper& h, hipStream_t st) {
  const dim3 grid((unsigned)b.count), block(kMuonSmall * kThreads);
  return sp == 16 ? launch_kernel(k_muon_small<1>, grid, block, st, b, h)
                  : launch_kernel(k_muon_small<2>, grid, block, st, b, h);
}

hipError_t launch_muon_poly(int count, int sp, const MuonHyper& h, const MuonScratch& s,
                            hipStream_t st) {
  const dim3 grid((unsigned)count);
  hipError_t e = hipSuccess;
  switch (sp) {
    case 16: return launch_kernel(k_muon_poly<1>, grid, dim3(64 * poly_waves(1)), st, h, s);
    case 32: return launch_kernel(k_muon_poly<2>, grid, dim3(64 * poly_waves(2)), st, h, s);
    case 64:
      e = launch_kernel(k_muon_sum<4>, dim3(10, (unsigned)count), dim3(kThreads), st, s);
      return e != hipSuccess ? e : launch_kernel(k_muon_poly64, grid, dim3(kPoly64), st, h, s);
    default:
      e = launch_kernel(k_muon_sum<8>, dim3(36, (unsigned)count), dim3(kThreads), st, s);
      return e != hipSuccess ? e : launch_kernel(k_muon_poly<8>, grid, dim3(64 * poly_waves(8)), st, h, s);
  }
}

hipError_t launch_muon_apply(int sp, int chunks, const MuonHyper& h, const MuonScratch& s,
                             hipStream_t st) {
  const dim3 grid((unsigned)chunks), block(kThreads);
  switch (sp) {
    case 16: return launch_kernel(k_muon_apply<1>, grid, block, st, h, s);
    case 32: return launch_kernel(k_muon_apply<2>, grid, block, st, h, s);
    case 64: return launch_kernel(k_muon_apply<4>, grid, block, st, h, s);
    default: return launch_kernel(k_muon_apply<8>, grid, block, st, h, s);
  }
}

}  // namespace qnf4
