// Activation checkpoints in 8 bits: what the backward of an adapted linear
// reads of its input is G^T X, so the input is kept as int8 codes with one
// float32 scale per 64 values of a row, and multiplied from that form.
//
//     a = max |x| of the block,  code = rint(127 x / a),  scale = fl(a / 127)
//
// 127 x is exact in float32 (a bf16 has 8 significant bits) and the quotient
// of a 15-bit by an 8-bit integer is never nearer than 2^-17 of itself to a
// half-integer unless it is one, so the code is the rounding (half to even)
// of the exact quotient whichever correctly rounded division forms it.
#include "grads.h"

namespace qnf4 {
namespace {

// Both directions move about three bytes a value with little to compute and
// are bound by HBM: 4096 x 22016 there and back in 91 us, 6.1 TB/s.  A
// workgroup takes 32 rows x 256 columns: 32 lanes hold a row's 256 values, 16
// bytes each, so every load and store instruction covers whole 256- to
// 1024-byte runs of two rows, a lane has its four rows' loads in flight
// together, and 8 neighbouring lanes hold one block, whose maximum is three DPP
// steps on packed 16-bit magnitudes.  32 rows are what makes the
// scales, which run along rows, whole 128-byte lines.
constexpr int kTileRows = 32, kTileCols = 256, kTileKb = kTileCols / kBlock;
constexpr int kRowsPerStep = 8;                     // 256 threads / 32 lanes a row
constexpr int kSteps = kTileRows / kRowsPerStep;

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                __builtin_bit_cast(u16x2_t, b)));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
}

// Largest magnitude (bf16 bits) of the 64 values 8 lanes hold, in all 8.  As
// integers the magnitudes order like the values, infinities and NaN on top.
__device__ __forceinline__ uint32_t block_max(const uint4& v) {
  constexpr uint32_t kMag = 0x7FFF7FFFu;
  uint32_t a = pk_max_u16(pk_max_u16(v.x & kMag, v.y & kMag), pk_max_u16(v.z & kMag, v.w & kMag));
  a = pk_max_u16(a, dpp_u32<kDppQuadXor1>(a));
  a = pk_max_u16(a, dpp_u32<kDppQuadXor2>(a));
  a = pk_max_u16(a, dpp_u32<kDppHalfMirror>(a));
  const uint32_t hi = a >> 16, lo = a & 0xFFFFu;
  return hi > lo ? hi : lo;
}

__global__ __launch_bounds__(256) void k_act8_quantize(const uint16_t* __restrict__ x,
                                                       int64_t rows, int64_t rows32, int64_t kb,
                                                       int64_t tiles_k, int8_t* __restrict__ codes,
                                                       float* __restrict__ scale) {
  __shared__ float sc[kTileKb][kTileRows];
  const int tid = threadIdx.x, l32 = tid & 31, rr = tid >> 5;
  const int64_t cols = kb * kBlock;
  const int64_t m0 = ((int64_t)blockIdx.x / tiles_k) * kTileRows;
  const int64_t kb0 = ((int64_t)blockIdx.x % tiles_k) * kTileKb;
  const int64_t c = kb0 * kBlock + 8 * l32;
  const bool in = c < cols;
  uint4 v[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t m = m0 + i * kRowsPerStep + rr;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (in && m < rows)
      v[i] = __builtin_bit_cast(uint4, __builtin_nontemporal_load(
                                           reinterpret_cast<const u32x4_t*>(x + m * cols + c)));
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t m = m0 + i * kRowsPerStep + rr;
    const uint32_t mag = block_max(v[i]);
    const bool bad = mag >= 0x7F80u;                  // an infinity or a NaN in the block
    const float a = bf16_to_f32((uint16_t)mag);
    // a power of two keeps 127 x, the reciprocal and the residual in range
    const float pre = a > 0x1p60f ? 0x1p-64f : (a < 0x1p-60f ? 0x1p64f : 1.f);
    const float b = a * pre;
    const bool some = !bad && mag != 0;
    float r = __builtin_amdgcn_rcpf(some ? b : 1.f);
    r = __builtin_fmaf(__builtin_fmaf(-b, r, 1.f), r, r);
    r = some ? r : 0.f;
    const float pre127 = bad ? 0.f : 127.f * pre;
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = (e & 1) ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16;
      const float n = bad ? 0.f : __builtin_bit_cast(float, h) * pre127;   // 127 x, exact
      // the quotient to within 2^-22, then its residual: a half-integer comes
      // out exact, and anything else is too far from one to cross it
      const float q0 = n * r;
      const float q1 = __builtin_fmaf(__builtin_fmaf(-b, q0, n), r, q0);
      q[e] = (uint32_t)(int)__builtin_rintf(q1);
    }
    uint2 out;
    out.x = (q[0] & 0xFFu) | ((q[1] & 0xFFu) << 8) | ((q[2] & 0xFFu) << 16) | (q[3] << 24);
    out.y = (q[4] & 0xFFu) | ((q[5] & 0xFFu) << 8) | ((q[6] & 0xFFu) << 16) | (q[7] << 24);
    if (in && m < rows) *reinterpret_cast<uint2*>(codes + m * cols + c) = out;
    if ((l32 & 7) == 0) sc[l32 >> 3][i * kRowsPerStep + rr] = bad ? __builtin_nanf("") : a / 127.f;
  }
  __syncthreads();
  // rows past the end held zeros, so their scales are the padding's zeros
  const int row = tid & 31, j = tid >> 5;
  if (j < kTileKb && kb0 + j < kb && m0 + row < rows32)
    scale[(kb0 + j) * rows32 + m0 + row] = sc[j][row];
}

template <bool BF16>
__global__ __launch_bounds__(256) void k_act8_dequantize(const int8_t* __restrict__ codes,
                                                         const float* __restrict__ scale,
                                                         int64_t rows, int64_t rows32, int64_t kb,
                                                         int64_t tiles_k, void* __restrict__ out) {
  const int tid = threadIdx.x, l32 = tid & 31, rr = tid >> 5;
  const int64_t cols = kb * kBlock;
  const int64_t m0 = ((int64_t)blockIdx.x / tiles_k) * kTileRows + rr;
  const int64_t c = ((int64_t)blockIdx.x % tiles_k) * kTileCols + 8 * l32;
  if (c >= cols) return;
  uint2 v[kSteps];
  float s[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    int64_t m = m0 + i * kRowsPerStep;
    m = m < rows ? m : rows - 1;
    v[i] = *reinterpret_cast<const uint2*>(codes + m * cols + c);
    s[i] = scale[(c / kBlock) * rows32 + m];
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t m = m0 + i * kRowsPerStep;
    if (m >= rows) return;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int w = (int)(e < 4 ? v[i].x : v[i].y);
      f[e] = (float)(w << (24 - 8 * (e & 3)) >> 24) * s[i];
    }
    if constexpr (BF16) {
      const u32x4_t o = {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                         pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
      __builtin_nontemporal_store(o, reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(out) +
                                                                m * cols + c));
    } else {
      f32x4_t* o = reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + m * cols + c);
      __builtin_nontemporal_store(f32x4_t{f[0], f[1], f[2], f[3]}, o);
      __builtin_nontemporal_store(f32x4_t{f[4], f[5], f[6], f[7]}, o + 1);
    }
  }
}

// ------------------------------------------------ adapter gradient from codes
//     partial[j][k] = sum_m (G[j][m] scale[kb][m]) code[m][k]
// on the matrix cores.  A code is exact in bf16, so the scale goes to the side
// of G: per block of 64 columns the 16 RT rows of G are multiplied by it
// instead of the 64 columns (less work up to rank 64), and only that product
// needs more than 8 bits.  It is cut into three bf16 parts by truncation,
// which together are the float32 value, and each part meets the same codes:
// three MFMAs where one would leave dA with bf16 errors (relative error 2e-7
// against 2e-3).  Bound by issue: 6.5 operations for each product of G and a
// scale and three MFMAs for each 16 x 16 x 32; at rank 16 the codes' way from
// memory shows first.  With dB in the same launch, codes of 4096 x 22016 and dY of
// 4096 x 8192 at rank 64 take 64 us, 2048 x 4096 and 2048 x 14336 at rank 16 13.5.
//
// A workgroup takes 128 columns (two blocks) of a token slice: waves 0 and 1 the
// even 32-token steps, waves 2 and 3 the odd ones, the second of each pair the
// second block (the pair reads the same rows of G, once from the L2).  Lane
// (i16, g) loads, for rows m = 8 g .. 8 g + 7 of a step, the 4 codes of columns
// 4 i16 .. 4 i16 + 3: MFMA t handles columns 4 i + t, and converting byte t of
// the eight rows is the transpose.  The next step's loads are in flight under a
// step's work; 64 columns a wave keep that within two waves' registers at four
// rank tiles, and ranks above 64 are two slices' work.  The token halves are
// added in order through LDS, 16 rank indices at a time, and leave as rows of
// 128 columns.
constexpr int kGradCols = 128, kGradTokens = 64;   // a workgroup's, per pass

template <int RT>
struct GradStep {
  uint32_t code[8];
  uint8_t keep[8];         // dropout's stored bits, unused without
  float4 scale[2];
  float4 g[RT][2];
};

__device__ __forceinline__ float elem(const float4 (&v)[2], int e) {
  const float4& q = v[e >> 2];
  return (e & 3) == 0 ? q.x : (e & 3) == 1 ? q.y : (e & 3) == 2 ? q.z : q.w;
}

// high halves of two words: b's above a's
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

__device__ __forceinline__ uint32_t nibble_mask(uint32_t n) {   // 4 keep bits -> 4 bytes
  return (((n & 1u) | ((n & 2u) << 7) | ((n & 4u) << 14) | ((n & 8u) << 21))) * 0xFFu;
}

template <int RT, bool DROP>
__device__ __forceinline__ void act8_grad_slice(const Act8GradJob& J, int64_t M, int r,
                                                int64_t block, int jt0, int rt) {
  __shared__ float red[2][16][kGradCols + 4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = wv >> 1, side = wv & 1;
  const int i16 = lane & 15, g = lane >> 4;
  const int split = (int)(block % J.splits);
  const int64_t p0 = (block / J.splits) * kGradCols;
  const int64_t mchunk = ceil_div(ceil_div(M, J.splits), kGradTokens) * kGradTokens;
  const int64_t mbeg = (int64_t)split * mchunk;
  int64_t mend = mbeg + mchunk;
  mend = mend < M ? mend : M;
  // a last workgroup of one block reads it twice and drops the second
  const int64_t blk = p0 / kBlock + (side && p0 + kBlock < J.K ? 1 : 0);

  f32x4_t acc[4][RT];
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int jt = 0; jt < RT; ++jt) acc[t][jt] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const bool bits = DROP && J.drop.bits;
  const uint32_t K = (uint32_t)J.K;
  // rows past M are clamped copies that meet G = 0 and scale = 0; mb + 31 is
  // inside ldg, a multiple of 32
  auto load = [&](int64_t mb, GradStep<RT>& s) {
    const int8_t* base = J.codes + mb * J.K + blk * kBlock;     // uniform
    const int64_t first = mb * J.K + blk * kBlock;
    const int left = (int)(M - 1 - mb < 31 ? M - 1 - mb : 31);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int row = 8 * g + e < left ? 8 * g + e : left;
      const uint32_t at = (uint32_t)row * K + 4 * i16;
      s.code[e] = *reinterpret_cast<const uint32_t*>(base + at);
      if constexpr (DROP)
        if (bits) s.keep[e] = J.drop.bits[(first + at) >> 3];
    }
    const float4* p = reinterpret_cast<const float4*>(J.scale + blk * J.ldg + mb) + 2 * g;
    s.scale[0] = p[0];
    s.scale[1] = p[1];
    // (a rank index past r feeds only rows of the partial that are never stored)
    const float4* q = reinterpret_cast<const float4*>(J.G) + ((mb >> 5) * rt + jt0) * 128;
#pragma unroll
    for (int jt = 0; jt < RT; ++jt) {
      s.g[jt][0] = q[(2 * jt) * 64 + lane];
      s.g[jt][1] = q[(2 * jt + 1) * 64 + lane];
    }
  };
  auto work = [&](int64_t mb, GradStep<RT>& s) {
    if constexpr (DROP) {
      const int64_t first = mb * J.K + blk * kBlock;
      const int left = (int)(M - 1 - mb < 31 ? M - 1 - mb : 31);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int row = 8 * g + e < left ? 8 * g + e : left;
        const uint64_t at = (uint64_t)(first + (uint32_t)row * K + 4 * i16);
        const uint32_t n = bits ? (uint32_t)s.keep[e] >> (at & 4)
                                : keep_nibble(dropout_words(at >> 2, J.drop), J.drop.thr);
        s.code[e] &= nibble_mask(n);
      }
    }
    uint4 a[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      uint32_t f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        f[e] = __builtin_bit_cast(uint32_t, (float)((int)(s.code[e] << (24 - 8 * t)) >> 24));
      a[t] = make_uint4(high_halves(f[0], f[1]), high_halves(f[2], f[3]),
                        high_halves(f[4], f[5]), high_halves(f[6], f[7]));
    }
#pragma unroll
    for (int jt = 0; jt < RT; ++jt) {
      uint32_t p1[8], p2[8], p3[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = elem(s.g[jt], e) * elem(s.scale, e);
        p1[e] = __builtin_bit_cast(uint32_t, v);
        const float rest = v - __builtin_bit_cast(float, p1[e] & 0xFFFF0000u);
        p2[e] = __builtin_bit_cast(uint32_t, rest);
        p3[e] = __builtin_bit_cast(uint32_t,
                                   rest - __builtin_bit_cast(float, p2[e] & 0xFFFF0000u));
      }
      auto operand = [](const uint32_t (&p)[8]) {
        return make_uint4(high_halves(p[0], p[1]), high_halves(p[2], p[3]),
                          high_halves(p[4], p[5]), high_halves(p[6], p[7]));
      };
      const uint4 b1 = operand(p1), b2 = operand(p2), b3 = operand(p3);
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t][jt] = mfma16x16x32(a[t], b3, acc[t][jt]);
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t][jt] = mfma16x16x32(a[t], b2, acc[t][jt]);
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t][jt] = mfma16x16x32(a[t], b1, acc[t][jt]);
    }
    // one rank tile's matrix instructions between the next one's arithmetic
    __builtin_amdgcn_sched_group_barrier(0x2, 100, 0);
#pragma unroll
    for (int k = 0; k < 12 * RT; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);
    }
  };
  const int64_t first = mbeg + 32 * half;
  const int64_t cnt = first < mend ? (mend - first + kGradTokens - 1) / kGradTokens : 0;
  auto step = [&](int64_t i) { return first + kGradTokens * i; };
  if (cnt > 0) {
    GradStep<RT> s0, s1;
    load(first, s0);
    int64_t i = 0;
    for (; i + 1 < cnt; i += 2) {
      load(step(i + 1), s1);
      __builtin_amdgcn_sched_barrier(0);
      work(step(i), s0);
      __builtin_amdgcn_sched_barrier(0);
      load(step(i + 2 < cnt ? i + 2 : i), s0);   // (after the last step: unused)
      __builtin_amdgcn_sched_barrier(0);
      work(step(i + 1), s1);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (i < cnt) work(step(i), s0);
  }
  // D[i = 4 g + v][j16] of MFMA t: column 16 g + 4 v + t of the wave's block
  float* base = J.partial + (int64_t)split * r * J.K + p0;
#pragma unroll
  for (int jt = 0; jt < RT; ++jt) {
    if (jt > 0) __syncthreads();
#pragma unroll
    for (int v = 0; v < 4; ++v)
      *reinterpret_cast<float4*>(&red[half][i16][64 * side + 16 * g + 4 * v]) =
          make_float4(acc[0][jt][v], acc[1][jt][v], acc[2][jt][v], acc[3][jt][v]);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int j = (tid >> 5) + 8 * q, p = 4 * (tid & 31);
      float4 s = *reinterpret_cast<const float4*>(&red[0][j][p]);
      const float4 o = *reinterpret_cast<const float4*>(&red[1][j][p]);
      s.x += o.x; s.y += o.y; s.z += o.z; s.w += o.w;
      if constexpr (DROP) {
        s.x *= J.drop.inv; s.y *= J.drop.inv; s.z *= J.drop.inv; s.w *= J.drop.inv;
      }
      const int rank = (jt0 + jt) * 16 + j;
      if (rank < r && p0 + p < J.K)
        *reinterpret_cast<float4*>(base + (int64_t)rank * J.K + p) = s;
    }
  }
}

// dA from the codes and dB from dY in one launch: neither needs the other, and
// one's last workgroups run beside the other's first.
template <int RT, bool DROP>
__global__ __launch_bounds__(256, 2) void k_act8_grads(Act8GradJob a, GradJob b, int64_t M,
                                                      int r) {
  const int parts = grad_parts(r);
  const int64_t block = blockIdx.x / parts, na = ceil_div(a.K, kGradCols) * a.splits;
  const int jt0 = (int)(blockIdx.x - block * parts) * RT, rt = RT * parts;
  if (block < na) act8_grad_slice<RT, DROP>(a, M, r, block, jt0, rt);
  else grad_slice<RT, false>(b, M, r, block - na, jt0, rt);
}

template <int RT>
hipError_t act8_grads_rt(const Act8GradJob& a, const GradJob& b, int64_t M, int r,
                         hipStream_t s) {
  const int64_t blocks =
      (ceil_div(a.K, kGradCols) * a.splits + grad_blocks(b)) * grad_parts(r);
  return launch_kernel(a.drop.thr != 0 ? k_act8_grads<RT, true> : k_act8_grads<RT, false>,
                       dim3((unsigned)blocks), dim3(256), s, a, b, M, r);
}

}  // namespace

int64_t act8_tiles(int64_t rows, int64_t cols) {
  return ceil_div(rows, kTileRows) * ceil_div(cols, kTileCols);
}

hipError_t launch_act8_quantize(const uint16_t* x, int64_t rows, int64_t cols, int8_t* codes,
                                float* scale, hipStream_t s) {
  const int64_t kb = cols / kBlock, rows32 = ceil_div(rows, 32) * 32;
  return launch_kernel(k_act8_quantize, dim3((unsigned)act8_tiles(rows, cols)), dim3(256), s, x,
                       rows, rows32, kb, ceil_div(cols, kTileCols), codes, scale);
}

hipError_t launch_act8_dequantize(const int8_t* codes, const float* scale, int64_t rows,
                                  int64_t cols, int bf16, void* out, hipStream_t s) {
  const int64_t kb = cols / kBlock, rows32 = ceil_div(rows, 32) * 32;
  return launch_kernel(bf16 ? k_act8_dequantize<true> : k_act8_dequantize<false>,
                       dim3((unsigned)act8_tiles(rows, cols)), dim3(256), s, codes, scale, rows,
                       rows32, kb, ceil_div(cols, kTileCols), out);
}

// About 192 workgroups (dB's fill the rest of the chip), at least two 32-token
// steps a wave.  More slices shorten the launch until the chip is full and then
// only add partials: with the reduction, 2048 x 4096 at rank 48 takes 40, 26,
// 20 and 22 us with 1, 2, 4 and 8 slices, 4096 x 22016 at rank 64 75, 73, 74
// and 82.
int act8_grad_splits(int64_t M, int64_t K) {
  int64_t splits = ceil_div(192, ceil_div(K, kGradCols));
  const int64_t maxs = ceil_div(M, 2 * kGradTokens);
  if (splits > maxs) splits = maxs;
  return (int)splits;
}

hipError_t launch_act8_grads(const Act8GradJob& a, const GradJob& b, int64_t M, int r,
                             hipStream_t s) {
  switch (skinny_rpad(r)) {
    case 16: return act8_grads_rt<1>(a, b, M, r, s);
    case 32: return act8_grads_rt<2>(a, b, M, r, s);
    default: return act8_grads_rt<4>(a, b, M, r, s);
  }
}

}  // namespace qnf4
