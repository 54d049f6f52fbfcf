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
#include "skinny.h"

namespace qnf4 {
namespace {

// Both directions move about three bytes a value with little to compute and
// are bound by HBM.  A workgroup takes 32 rows x 256 columns: 32 lanes hold a
// row's 256 values, 16 bytes each, so every load and store instruction covers
// whole 256- to 1024-byte runs of two rows, a lane has its four rows' loads
// in flight together, and 8 neighbouring lanes hold one block, whose maximum
// is three DPP steps on packed 16-bit magnitudes.  32 rows are what makes the
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

// Thread per column p and eight rank indices: dA[j][p] = scale inv sum_m
// G[j][m] keep(m, p) scale[m] code[m][p].
__global__ __launch_bounds__(256) void k_act8_grad(Act8GradJob J, int64_t M, int r) {
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int j0 = blockIdx.y * 8;
  if (p >= J.K) return;
  float acc[8] = {};
  for (int64_t m = 0; m < M; ++m) {
    float v = (float)J.codes[m * J.K + p] * J.scale[(p / kBlock) * J.ldg + m];
    if (J.drop.thr != 0) {
      const uint64_t e = (uint64_t)(m * J.K + p);
      v = (dropout_byte(e & ~7ull, J.drop) >> (e & 7)) & 1u ? v : 0.f;
    }
    for (int j = 0; j < 8; ++j)
      if (j0 + j < r) acc[j] = __builtin_fmaf(J.G[(int64_t)(j0 + j) * J.ldg + m], v, acc[j]);
  }
  for (int j = 0; j < 8; ++j)
    if (j0 + j < r) J.out[(int64_t)(j0 + j) * J.K + p] = J.alpha * (J.drop.inv * acc[j]);
}

}  // namespace

hipError_t launch_act8_quantize(const uint16_t* x, int64_t rows, int64_t cols, int8_t* codes,
                                float* scale, hipStream_t s) {
  const int64_t kb = cols / kBlock, rows32 = ceil_div(rows, 32) * 32;
  const int64_t tk = ceil_div(cols, kTileCols);
  return launch_kernel(k_act8_quantize, dim3((unsigned)(tk * (rows32 / kTileRows))), dim3(256), s,
                       x, rows, rows32, kb, tk, codes, scale);
}

hipError_t launch_act8_dequantize(const int8_t* codes, const float* scale, int64_t rows,
                                  int64_t cols, int bf16, void* out, hipStream_t s) {
  const int64_t kb = cols / kBlock, rows32 = ceil_div(rows, 32) * 32;
  const int64_t tk = ceil_div(cols, kTileCols);
  return launch_kernel(bf16 ? k_act8_dequantize<true> : k_act8_dequantize<false>,
                       dim3((unsigned)(tk * (rows32 / kTileRows))), dim3(256), s, codes, scale,
                       rows, rows32, kb, tk, out);
}

hipError_t launch_act8_grad(const Act8GradJob& job, int64_t M, int r, hipStream_t s) {
  return launch_kernel(k_act8_grad, dim3((unsigned)ceil_div(job.K, 256), (unsigned)ceil_div(r, 8)),
                       dim3(256), s, job, M, r);
}

}  // namespace qnf4
