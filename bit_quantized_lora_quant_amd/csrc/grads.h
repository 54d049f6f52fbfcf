// Adapter gradients from bf16 rows as one slice of a workgroup: shared by the
// plain backward's launch and the one that reads 8-bit checkpoints.
#pragma once

#include "skinny.h"

namespace qnf4 {

constexpr int kGradP = 64;   // columns of a workgroup

// Raw 8-byte load of a buffer view (buffer_load16 of skinny.h).
__device__ __forceinline__ uint2 buffer_load8(__amdgpu_buffer_rsrc_t v, uint32_t lane_off,
                                              uint32_t uniform_off) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(v, (int)lane_off,
                                                                        (int)uniform_off, 0));
}
// 4 consecutive bf16 at p[idx ..]; entries at or past `limit` read 0
__device__ __forceinline__ uint2 load4_bf16(const uint16_t* __restrict__ p, int64_t idx,
                                            int64_t limit) {
  uint16_t e[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) e[q] = (idx + q < limit) ? p[idx + q] : (uint16_t)0;
  return make_uint2(e[0] | ((uint32_t)e[1] << 16), e[2] | ((uint32_t)e[3] << 16));
}

// Workgroup (64 consecutive p, token slice): the 4 waves take interleaved
// 32-token steps.  Lane (i16, g) loads 8 rows m (8g..8g+7 of a step) x 4
// consecutive p (4 i16 .. 4 i16 + 3) of T and regroups them into the A
// operands of 4 MFMAs: MFMA t handles p = p0 + 4 i + t, so the transpose of T
// costs one 16-bit regroup per pair of rows, no LDS.  64 columns leave two
// waves a SIMD their registers with two steps in flight each (128 columns left
// one: 4096 x 8192 at rank 64 27 us, now 22.6).  Wave partials are added in
// wave order through LDS, one MFMA column t at a time.  With DROP, a job whose
// J.drop is set reads T = X through the dropout mask and scales its partials by
// J.drop.inv.
// RT rank tiles from tile jt0 on, of rt in all: above rank 64 the tiles are two
// slices' work (2048 x 4096 at rank 128 21 us, 31 as one slice of eight tiles).
template <int RT, bool DROP>
__device__ __forceinline__ void grad_slice(const GradJob& J, int64_t M, int r, int64_t b,
                                           int jt0 = 0, int rt = RT) {
  __shared__ float red[4][RT][4][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);   // wave-uniform
  const int i16 = lane & 15, g = lane >> 4;
  const int split = (int)(b % J.splits);
  const int64_t p0 = (b / J.splits) * kGradP;
  const int64_t mchunk = ceil_div(ceil_div(M, J.splits), 32) * 32;
  const int64_t mbeg = (int64_t)split * mchunk;
  int64_t mend = mbeg + mchunk;
  mend = mend < M ? mend : M;
  // rows of whole groups of 4 columns are read as such, a last tile's lanes past
  // them repeating the row's last group: what they make is never stored
  const bool fast = (J.P % 4) == 0;
  const int64_t pc = fast && p0 + 4 * i16 >= J.P ? J.P - 4 : p0 + 4 * i16;

  f32x4_t acc[4][RT];
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int jt = 0; jt < RT; ++jt) acc[t][jt] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // step mb: rows mb + 8g + e of T (clamped below M; U is zero there) and the
  // fragments of U.  A rank index past r feeds only output column j >= r, which
  // is never stored, so what its slots hold does not matter.
  auto load_step = [&](int64_t mb, uint2 (&rows)[8], uint4 (&bu)[RT]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      int64_t m = mb + 8 * g + e;
      m = m < M ? m : M - 1;
      if (fast) rows[e] = *reinterpret_cast<const uint2*>(J.T + m * J.P + pc);
      else rows[e] = load4_bf16(J.T + m * J.P, pc, J.P);
    }
#pragma unroll
    for (int jt = 0; jt < RT; ++jt)
      bu[jt] = *reinterpret_cast<const uint4*>(J.U + ((mb >> 5) * rt + jt0 + jt) * 512 + lane * 8);
  };
  auto mfmas = [&](const uint2 (&rows)[8], const uint4 (&bu)[RT]) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      uint32_t h[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t w = t < 2 ? rows[e].x : rows[e].y;
        h[e] = (t & 1) ? (w >> 16) : (w & 0xFFFFu);
      }
      uint4 a;
      a.x = h[0] | (h[1] << 16);
      a.y = h[2] | (h[3] << 16);
      a.z = h[4] | (h[5] << 16);
      a.w = h[6] | (h[7] << 16);
#pragma unroll
      for (int jt = 0; jt < RT; ++jt) acc[t][jt] = mfma16x16x32(a, bu[jt], acc[t][jt]);
    }
  };
  // dropout of T's rows of step mb (wave-uniform switch); rows past M are
  // clamped copies that meet zero columns of U
  const bool dj = DROP && J.drop.thr != 0;
  auto drop_t = [&](int64_t mb, uint2 (&rows)[8]) {
    if constexpr (DROP) {
      if (dj) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          int64_t m = mb + 8 * g + e;
          m = m < M ? m : M - 1;
          const uint64_t at = (uint64_t)m * (uint64_t)J.drop.cols + pc;
          const uint32_t n = J.drop.bits ? (uint32_t)J.drop.bits[at >> 3] >> (at & 4)
                                         : keep_nibble(dropout_words(at >> 2, J.drop), J.drop.thr);
          const uint4 k = byte_mask8(n);
          rows[e].x &= k.x;
          rows[e].y &= k.y;
        }
      }
    }
  };
  // this wave's steps: mb = first + 128 i, i < cnt
  const int64_t first = mbeg + 32 * wv;
  const int64_t cnt = first < mend ? (mend - first + 127) / 128 : 0;
  // Steps of 32 whole rows of such groups read through buffer views
  // (fixed byte offsets per lane, the step's base as the uniform offset), two
  // steps in flight: the next step's loads are issued before this step's MFMAs.
  const int64_t tbytes = M * J.P * 2, ubytes = ceil_div(M, 32) * rt * 1024;
  const bool bufs = fast && tbytes <= kBufferMax && ubytes <= kBufferMax;
  const int64_t cnt_fast = bufs && first + 32 <= mend ? (mend - first - 32) / 128 + 1 : 0;
  if (cnt_fast > 0) {
    const __amdgpu_buffer_rsrc_t tview = buffer_view(J.T, tbytes);
    const __amdgpu_buffer_rsrc_t uview = buffer_view(J.U, ubytes);
    uint32_t roff[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) roff[e] = (uint32_t)((8 * g + e) * J.P + pc) * 2;
    auto load_fast = [&](int64_t i, uint2 (&rows)[8], uint4 (&bu)[RT]) {
      const int64_t mb = first + 128 * i;
      const uint32_t tb = (uint32_t)(mb * J.P) * 2, ub = (uint32_t)(mb >> 5) * (rt * 1024);
#pragma unroll
      for (int e = 0; e < 8; ++e) rows[e] = buffer_load8(tview, roff[e], tb);
#pragma unroll
      for (int jt = 0; jt < RT; ++jt)
        bu[jt] = buffer_load16(uview, lane * 16 + (jt0 + jt) * 1024, ub);
    };
    uint2 r0[8], r1[8];
    uint4 u0[RT], u1[RT];
    load_fast(0, r0, u0);
    int64_t i = 0;
    for (; i + 2 < cnt_fast; i += 2) {
      load_fast(i + 1, r1, u1);
      __builtin_amdgcn_sched_barrier(0);
      drop_t(first + 128 * i, r0);
      mfmas(r0, u0);
      __builtin_amdgcn_sched_barrier(0);
      load_fast(i + 2, r0, u0);
      __builtin_amdgcn_sched_barrier(0);
      drop_t(first + 128 * (i + 1), r1);
      mfmas(r1, u1);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (i + 1 < cnt_fast) {   // the last one or two steps, peeled
      load_fast(i + 1, r1, u1);
      __builtin_amdgcn_sched_barrier(0);
      drop_t(first + 128 * i, r0);
      mfmas(r0, u0);
      __builtin_amdgcn_sched_barrier(0);
      drop_t(first + 128 * (i + 1), r1);
      mfmas(r1, u1);
    } else {
      drop_t(first + 128 * i, r0);
      mfmas(r0, u0);
    }
  }
  // the rest (a last step of fewer rows, or ragged columns): one step at a
  // time, rows clamped
  for (int64_t i = cnt_fast; i < cnt; ++i) {
    uint2 r0[8];
    uint4 u0[RT];
    load_step(first + 128 * i, r0, u0);
    drop_t(first + 128 * i, r0);
    mfmas(r0, u0);
  }
  // D[i = 4g + v][j16] of MFMA (t, jt): p = p0 + 4 (4g + v) + t, j = 16 jt + j16
  float* base = J.partial + (int64_t)split * J.P * r;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
#pragma unroll
    for (int jt = 0; jt < RT; ++jt)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[wv][jt][v][lane] = acc[t][jt][v];
    __syncthreads();
    if (wv == t) {
#pragma unroll
      for (int jt = 0; jt < RT; ++jt)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float s = red[0][jt][v][lane];
#pragma unroll
          for (int w = 1; w < 4; ++w) s += red[w][jt][v][lane];
          if constexpr (DROP) s *= J.drop.inv;
          const int64_t p = p0 + 4 * (4 * g + v) + t;
          const int j = (jt0 + jt) * 16 + i16;
          // partials in the output's own layout, so the reduce reads them
          // contiguously
          if (p < J.P && j < r) base[J.transposed ? (int64_t)j * J.P + p : p * r + j] = s;
        }
    }
    __syncthreads();
  }
}

// Slices' worth of rank tiles.
__host__ __device__ __forceinline__ int grad_parts(int r) { return r > 64 ? 2 : 1; }

__host__ __device__ __forceinline__ int64_t grad_blocks(const GradJob& J) {
  return ceil_div(J.P, kGradP) * J.splits;
}

}  // namespace qnf4
