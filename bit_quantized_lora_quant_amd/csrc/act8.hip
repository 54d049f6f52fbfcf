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

// Thread per block of 64.
__global__ __launch_bounds__(256) void k_act8_quantize(const uint16_t* __restrict__ x,
                                                       int64_t rows, int64_t rows32, int64_t kb,
                                                       int8_t* __restrict__ codes,
                                                       float* __restrict__ scale) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= rows32 * kb) return;
  const int64_t m = i / kb, b = i - m * kb;
  if (m >= rows) {
    scale[b * rows32 + m] = 0.f;
    return;
  }
  const uint16_t* p = x + (m * kb + b) * kBlock;
  float a = 0.f;
  bool bad = false;
  for (int e = 0; e < kBlock; ++e) {
    const float v = __builtin_fabsf(bf16_to_f32(p[e]));
    bad |= !(v < __builtin_inff());
    a = fmaxf(a, v);
  }
  // a power of two keeps 127 x and the reciprocal in range
  const float pre = a > 0x1p60f ? 0x1p-64f : (a < 0x1p-60f ? 0x1p64f : 1.f);
  for (int e = 0; e < kBlock; ++e) {
    const float q = bad || a == 0.f ? 0.f
                                    : __builtin_rintf(127.f * (bf16_to_f32(p[e]) * pre) / (a * pre));
    codes[(m * kb + b) * kBlock + e] = (int8_t)q;
  }
  scale[b * rows32 + m] = bad ? __builtin_nanf("") : a / 127.f;
}

__global__ __launch_bounds__(256) void k_act8_dequantize(const int8_t* __restrict__ codes,
                                                         const float* __restrict__ scale,
                                                         int64_t rows, int64_t rows32, int64_t kb,
                                                         int bf16, void* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= rows * kb) return;
  const int64_t m = i / kb, b = i - m * kb;
  const float s = scale[b * rows32 + m];
  for (int e = 0; e < kBlock; ++e) {
    const float v = (float)codes[i * kBlock + e] * s;
    if (bf16) static_cast<uint16_t*>(out)[i * kBlock + e] = to_bf16(v);
    else static_cast<float*>(out)[i * kBlock + e] = v;
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
  return launch_kernel(k_act8_quantize, dim3((unsigned)ceil_div(rows32 * kb, 256)), dim3(256), s,
                       x, rows, rows32, kb, codes, scale);
}

hipError_t launch_act8_dequantize(const int8_t* codes, const float* scale, int64_t rows,
                                  int64_t cols, int bf16, void* out, hipStream_t s) {
  const int64_t kb = cols / kBlock, rows32 = ceil_div(rows, 32) * 32;
  return launch_kernel(k_act8_dequantize, dim3((unsigned)ceil_div(rows * kb, 256)), dim3(256), s,
                       codes, scale, rows, rows32, kb, bf16, out);
}

hipError_t launch_act8_grad(const Act8GradJob& job, int64_t M, int r, hipStream_t s) {
  return launch_kernel(k_act8_grad, dim3((unsigned)ceil_div(job.K, 256), (unsigned)ceil_div(r, 8)),
                       dim3(256), s, job, M, r);
}

}  // namespace qnf4
