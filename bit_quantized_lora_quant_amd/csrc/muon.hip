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
//   k_muon_apply  workgroup per slice: O = Q U, then the parameter's update
//
// Bound: HBM for rank up to 64 (a step moves 30 bytes a parameter, 22 of them
// unavoidable: gradient and momentum are read again); the f64 matrix cores at 128.
#include "muon.h"

namespace qnf4 {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;        // groups of 4 neighbours per thread and chunk
constexpr int kBuf = 4096 + 4 * 128;   // floats of a chunk: sp rows of C + 4

typedef double f64x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f64x4_t mfma64(double a, double b, f64x4_t c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

// The workgroup's tensor seen along its short side s (index i) and long side n
// (index l): element (i, l) lies at i ld + l of a wide matrix, l ld + i of a tall one.
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

// Units of a chunk: 4 neighbours in memory, wide (C / 4 a row of s), tall
// (ceil(s / 4) a long index).  Unit u: short index, long index within the chunk.
struct Unit {
  int i, l;
};
__device__ __forceinline__ Unit unit_at(const View& v, int u) {
  if (v.tall) {
    const int per = (v.s + 3) / 4;
    return Unit{4 * (u % per), u / per};
  }
  const int per = v.chunk / 4;
  return Unit{u / per, 4 * (u % per)};
}
__device__ __forceinline__ int units(const View& v) {
  return v.tall ? v.chunk * ((v.s + 3) / 4) : v.s * (v.chunk / 4);
}
// How many of a unit's four elements there are.
__device__ __forceinline__ int unit_valid(const View& v, const Unit& a, int l0) {
  if (v.tall) return l0 + a.l < v.n ? (v.s - a.i < 4 ? v.s - a.i : 4) : 0;
  const int left = v.n - l0 - a.l;
  return left < 0 ? 0 : left < 4 ? left : 4;
}
__device__ __forceinline__ int64_t unit_off(const View& v, const Unit& a, int l0, int ld) {
  return v.tall ? (int64_t)(l0 + a.l) * ld + a.i : (int64_t)a.i * ld + l0 + a.l;
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

// A chunk of U lies in LDS as [short][long] with C + 4 floats a row: the 16 x 4
// operand reads and both kinds of writes meet each bank evenly.
__device__ __forceinline__ void put(float* u, const View& v, const Unit& a, const float (&x)[4]) {
  const int pitch = v.chunk + 4;
  if (v.tall) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (a.i + e < v.s) u[(a.i + e) * pitch + a.l] = x[e];
  } else {
    *reinterpret_cast<float4*>(u + a.i * pitch + a.l) = make_float4(x[0], x[1], x[2], x[3]);
  }
}
__device__ __forceinline__ void get(float (&x)[4], const float* u, const View& v, const Unit& a) {
  const int pitch = v.chunk + 4;
  if (v.tall) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = a.i + e < v.s ? u[(a.i + e) * pitch + a.l] : 0.f;
  } else {
    const float4 f = *reinterpret_cast<const float4*>(u + a.i * pitch + a.l);
    x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
  }
}
// rows past the short side: read by the matrix cores, never written after
__device__ __forceinline__ void clear_pad(float* u, const View& v) {
  const int pitch = v.chunk + 4;
  for (int k = v.s * pitch + threadIdx.x; k < v.sp * pitch; k += kThreads) u[k] = 0.f;
}

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
// wave takes every fourth product and all steps.
template <int NT>
struct Gram {
  static constexpr int kTiles = NT * (NT + 1) / 2;
  static constexpr bool kByStep = NT <= 2;
  static constexpr int kMine = kByStep ? kTiles : (kTiles + 3) / 4;
  f64x4_t acc[kMine];
  __device__ __forceinline__ void init() {
#pragma unroll
    for (int k = 0; k < kMine; ++k) acc[k] = f64x4_t{0., 0., 0., 0.};
  }
  __device__ __forceinline__ void add(const float* u, int lane, int wv) {
    constexpr int C = 4096 / (16 * NT), pitch = C + 4;
    const float* at = u + (lane & 15) * pitch + (lane >> 4);
    if (kByStep) {
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
#pragma unroll 2
      for (int l = 0; l < C; l += 4) {
        double x[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) x[i] = (double)at[i * 16 * pitch + l];
        // product k is wave k % 4's
        int k = 0;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = i; j < NT; ++j, ++k)
            if ((k & 3) == wv) acc[k >> 2] = mfma64(x[i], x[j], acc[k >> 2]);
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

template <int NT>
__device__ __forceinline__ void gram(const MuonTensor& t, const View& v, const MuonHyper& h,
                                     int slice, double* out, float* u, double* buf) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = slice * t.slice, end = first + t.slice < v.n ? first + t.slice : v.n;
  const int count = units(v);
  const bool vi = fits16(t.in, t.ldi, t.bf16 ? 2 : 4), vm = fits16(t.m, t.ldm, 4);
  float g[kUnits][4], m[kUnits][4];
  auto load = [&](int l0) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int id = threadIdx.x + k * kThreads;
      if (id >= count) break;
      const Unit a = unit_at(v, id);
      const int valid = unit_valid(v, a, l0);
      load_in(g[k], t, unit_off(v, a, l0, t.ldi), valid, vi);
      if (t.m) load4(m[k], t.m + unit_off(v, a, l0, t.ldm), valid, vm);
    }
  };
  Gram<NT> G;
  G.init();
  clear_pad(u, v);
  load(first);
  for (int l0 = first; l0 < end; l0 += v.chunk) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int id = threadIdx.x + k * kThreads;
      if (id >= count) break;
      const Unit a = unit_at(v, id);
      if (t.m) {
#pragma unroll
        for (int e = 0; e < 4; ++e) m[k][e] = momentum(m[k][e], g[k][e], h);
        store4(t.m + unit_off(v, a, l0, t.ldm), m[k], unit_valid(v, a, l0), vm);
#pragma unroll
        for (int e = 0; e < 4; ++e) g[k][e] = update(m[k][e], g[k][e], h);
      }
      put(u, v, a, g[k]);
    }
    __syncthreads();
    if (l0 + v.chunk < end) load(l0 + v.chunk);   // in flight under the products
    G.add(u, lane, wv);
    __syncthreads();
  }
  G.store(out, buf, lane, wv);
}

// (a launch per padded rank that the batch has: workgroups of another return)
template <int NT>
__global__ __launch_bounds__(kThreads) void k_muon_gram(const MuonBatch bt, MuonHyper h,
                                                        MuonScratch s) {
  __shared__ __attribute__((aligned(16))) float u[kBuf];
  __shared__ __attribute__((aligned(32))) double buf[NT <= 2 ? 3 * Gram<NT>::kTiles * 256 : 1];
  const int lane = threadIdx.x & 63;
  const int wg = bt.t[0].wg + blockIdx.x;
  const uint64_t before =
      __builtin_amdgcn_ballot_w64(lane < bt.count && bt.t[lane < bt.count ? lane : 0].wg <= wg);
  const int i = __builtin_amdgcn_readfirstlane(__popcll(before)) - 1;
  const MuonTensor t = bt.t[i];
  const View v = view(t);
  if (v.sp != 16 * NT) return;
  const int slice = wg - t.wg;
  if (threadIdx.x == 0) {
    s.owner[wg] = bt.first + i;
    if (slice == 0) s.t[bt.first + i] = t;
  }
  gram<NT>(t, v, h, slice, s.part + ((size_t)t.part + (size_t)slice * Gram<NT>::kTiles) * 256, u,
           buf);
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
__device__ __forceinline__ void put_panel(double* x, const Panel<NT>& p, int lane, int wv) {
  constexpr int pitch = 16 * NT + 2;
  double* at = x + (lane >> 4) * pitch + 16 * wv + (lane & 15);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) at[(16 * i + 4 * v) * pitch] = p.t[i][v];
  __syncthreads();
}

template <int NT>
__global__ __launch_bounds__(64 * NT) void k_muon_poly(MuonHyper h, MuonScratch s) {
  constexpr int pitch = 16 * NT + 2;
  __shared__ __attribute__((aligned(16))) double x[16 * NT * pitch];
  const MuonTensor t = s.t[blockIdx.x];
  const View vw = view(t);
  if (vw.sp != 16 * NT) return;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slices = (int)ceil_div(vw.n, t.slice), tiles = muon_tiles(vw.sp);
  // the slices' parts in order, both halves of the matrix
  int k = 0;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = i; j < NT; ++j, ++k) {
      if (k % NT != wv) continue;
      const f64x4_t* from = reinterpret_cast<const f64x4_t*>(s.part + ((size_t)t.part + k) * 256) + lane;
      f64x4_t g = f64x4_t{0., 0., 0., 0.};
#pragma unroll 8
      for (int p = 0; p < slices; ++p) g += from[(size_t)p * tiles * 64];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = 16 * i + 4 * v + (lane >> 4), c = 16 * j + (lane & 15);
        x[r * pitch + c] = g[v];
        x[c * pitch + r] = g[v];
      }
    }
  __syncthreads();
  double tr = 0;
  for (int r = lane; r < 16 * NT; r += 64) tr += x[r * (pitch + 1)];
#pragma unroll
  for (int d = 32; d; d >>= 1) tr += __shfl_xor(tr, d);
  const double norm = fmax(sqrt(tr), h.eps), inv = 1.0 / norm;
  // (fmax drops a NaN: then every product shows it)
  Panel<NT> G, Q;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v)
      G.t[i][v] = x[(16 * i + 4 * v + (lane >> 4)) * pitch + 16 * wv + (lane & 15)] * inv * inv;
  put_panel<NT>(x, G, lane, wv);
  for (int n = 0; n < h.steps; ++n) {
    Panel<NT> P = times<NT>(x, G, lane);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        P.t[i][v] = h.b * G.t[i][v] + h.c * P.t[i][v];
        if (i == wv && 4 * v + (lane >> 4) == (lane & 15)) P.t[i][v] += h.a;
      }
    const bool last = n + 1 == h.steps;
    Panel<NT> U;
    if (!last) U = times<NT>(x, P, lane);          // G P
    put_panel<NT>(x, P, lane, wv);
    if (n == 0) Q = P;
    else Q = times<NT>(x, Q, lane);                // P Q
    if (!last) {
      G = times<NT>(x, U, lane);                   // P G P
      put_panel<NT>(x, G, lane, wv);
    }
  }
  double* out = s.q + (size_t)t.q * 256 + (lane >> 4) * 16 * NT + 16 * wv + (lane & 15);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) out[(16 * i + 4 * v) * 16 * NT] = Q.t[i][v] * inv;
}

// --------------------------------------------------------------------- apply
// O = Q U of a chunk: wave w takes row tiles and columns so that its part of Q stays
// in registers over the whole slice.
template <int NT>
__device__ __forceinline__ void apply(const MuonTensor& t, const View& v, const MuonHyper& h,
                                      int slice, const double* q, float* u) {
  constexpr int SP = 16 * NT, C = 4096 / SP, pitch = C + 4;
  constexpr int RW = NT < 4 ? NT : 4;         // waves along the short side
  constexpr int MI = NT / RW;                 // row tiles of a wave
  constexpr int CW = 4 / RW;                  // waves along the long side
  constexpr int MJ = C / 16 / CW;             // column tiles of a wave
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wv % RW, wc = wv / RW;
  const int first = slice * t.slice, end = first + t.slice < v.n ? first + t.slice : v.n;
  const int count = units(v);
  const bool vi = fits16(t.in, t.ldi, t.bf16 ? 2 : 4), vm = fits16(t.m, t.ldm, 4);
  const bool vo = fits16(t.out, t.ldo, !h.step && t.bf16 ? 2 : 4), vb = fits16(t.pb, t.ldb, 2);
  const bool need_in = !t.m || h.nesterov;
  double a[MI][4 * NT];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int k = 0; k < 4 * NT; ++k)
      a[i][k] = q[(16 * (wr * MI + i) + (lane & 15)) * SP + 4 * k + (lane >> 4)];
  float g[kUnits][4], m[kUnits][4], p[kUnits][4];
  auto load = [&](int l0) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int id = threadIdx.x + k * kThreads;
      if (id >= count) break;
      const Unit b = unit_at(v, id);
      const int valid = unit_valid(v, b, l0);
      if (need_in) load_in(g[k], t, unit_off(v, b, l0, t.ldi), valid, vi);
      if (t.m) load4(m[k], t.m + unit_off(v, b, l0, t.ldm), valid, vm);
      if (h.step) load4(p[k], static_cast<const float*>(t.out) + unit_off(v, b, l0, t.ldo), valid, vo);
    }
  };
  clear_pad(u, v);
  for (int l0 = first; l0 < end; l0 += v.chunk) {
    load(l0);
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int id = threadIdx.x + k * kThreads;
      if (id >= count) break;
      if (t.m) {
#pragma unroll
        for (int e = 0; e < 4; ++e) g[k][e] = update(m[k][e], g[k][e], h);
      }
      put(u, v, unit_at(v, id), g[k]);
    }
    __syncthreads();
    f64x4_t o[MI][MJ];
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      const float* at = u + (lane >> 4) * pitch + 16 * (wc * MJ + j) + (lane & 15);
#pragma unroll
      for (int i = 0; i < MI; ++i) o[i][j] = f64x4_t{0., 0., 0., 0.};
#pragma unroll
      for (int k = 0; k < 4 * NT; ++k) {
        const double x = (double)at[4 * k * pitch];
#pragma unroll
        for (int i = 0; i < MI; ++i) o[i][j] = mfma64(a[i][k], x, o[i][j]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < MJ; ++j)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * (wr * MI + i) + 4 * r + (lane >> 4);
          if (row < v.s) u[row * pitch + 16 * (wc * MJ + j) + (lane & 15)] = (float)o[i][j][r];
        }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int id = threadIdx.x + k * kThreads;
      if (id >= count) break;
      const Unit b = unit_at(v, id);
      const int valid = unit_valid(v, b, l0);
      const int64_t off = unit_off(v, b, l0, t.ldo);
      float x[4];
      get(x, u, v, b);
      if (!h.step) {
        if (t.bf16) store4(static_cast<uint16_t*>(t.out) + off, x, valid, vo);
        else store4(static_cast<float*>(t.out) + off, x, valid, vo);
        continue;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = p[k][e] * h.decay - t.scale * x[e];
      store4(static_cast<float*>(t.out) + off, x, valid, vo);
      if (t.pb) store4(t.pb + unit_off(v, b, l0, t.ldb), x, valid, vb);
    }
    __syncthreads();
  }
}

// Last workgroups first: what the first launches read last is still in the
// Infinity Cache.
template <int NT>
__global__ __launch_bounds__(kThreads) void k_muon_apply(MuonHyper h, MuonScratch s) {
  __shared__ __attribute__((aligned(16))) float u[kBuf];
  const int wg = gridDim.x - 1 - blockIdx.x;
  const MuonTensor t = s.t[__builtin_amdgcn_readfirstlane(s.owner[wg])];
  const View v = view(t);
  if (v.sp != 16 * NT) return;
  apply<NT>(t, v, h, wg - t.wg, s.q + (size_t)t.q * 256, u);
}

}  // namespace

int muon_slice(int sp, int64_t total) {
  // at least 512 workgroups where there is work for them, at most 16 chunks (the
  // parts of a rank of 128 are as large as 4.5 chunks of it)
  const int64_t most = sp <= 32 ? 4 : sp == 64 ? 8 : 16;
  int64_t chunks = ceil_div(total, 512 * 4096);
  chunks = chunks < 1 ? 1 : chunks > most ? most : chunks;
  return (int)chunks * muon_chunk(sp);
}

hipError_t launch_muon_gram(const MuonBatch& b, int sp, int wgs, const MuonHyper& h,
                            const MuonScratch& s, hipStream_t st) {
  const dim3 grid((unsigned)wgs), block(kThreads);
  switch (sp) {
    case 16: return launch_kernel(k_muon_gram<1>, grid, block, st, b, h, s);
    case 32: return launch_kernel(k_muon_gram<2>, grid, block, st, b, h, s);
    case 64: return launch_kernel(k_muon_gram<4>, grid, block, st, b, h, s);
    default: return launch_kernel(k_muon_gram<8>, grid, block, st, b, h, s);
  }
}

hipError_t launch_muon_poly(int count, int sp, const MuonHyper& h, const MuonScratch& s,
                            hipStream_t st) {
  const dim3 grid((unsigned)count);
  switch (sp) {
    case 16: return launch_kernel(k_muon_poly<1>, grid, dim3(64), st, h, s);
    case 32: return launch_kernel(k_muon_poly<2>, grid, dim3(128), st, h, s);
    case 64: return launch_kernel(k_muon_poly<4>, grid, dim3(256), st, h, s);
    default: return launch_kernel(k_muon_poly<8>, grid, dim3(512), st, h, s);
  }
}

hipError_t launch_muon_apply(int sp, int wgs, const MuonHyper& h, const MuonScratch& s,
                             hipStream_t st) {
  const dim3 grid((unsigned)wgs), block(kThreads);
  switch (sp) {
    case 16: return launch_kernel(k_muon_apply<1>, grid, block, st, h, s);
    case 32: return launch_kernel(k_muon_apply<2>, grid, block, st, h, s);
    case 64: return launch_kernel(k_muon_apply<4>, grid, block, st, h, s);
    default: return launch_kernel(k_muon_apply<8>, grid, block, st, h, s);
  }
}

}  // namespace qnf4
