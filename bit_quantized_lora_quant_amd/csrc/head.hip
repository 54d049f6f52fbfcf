// The language-model head without its logits: log-probabilities and cross entropy
// from hidden states h [rows, D] and the head's weight W [V, D], both bf16.
//
//   z_t = W h_t,  logp_t = z_ty - log sum_v exp(z_tv)
//   dz_tv = w_t (1[v = y_t] - p_tv),  dh = dz W,  dW = dz^T h
//
// Rows with a target are packed first, so prompts and padding cost nothing and
// whatever they hold reaches no sum.  The packed rows go through in panels of at
// most 2^29 row x vocabulary elements.  The product's tiles leave, per row and slice
// of 128 vocabulary entries, the largest logit m and, with the whole exponent
// M = ceil(m log2 e), the sum of 2^(z log2 e - M).  The target is left out of its
// slice: its logit is a float64 dot
// product of the packing, and 1 - p of a nearly certain target is a sum of what is
// left, not 1 minus something rounded.  The slices are joined in float64, by powers
// of two only.
//
// A gradient in the same call has the slices' values written in 16 bits.  dh alone
// takes them as bf16, the matrix cores' type: its tile loop lowers their exponents
// by R - M to the row's R, and the row's factor and its target's term come in float32
// at the end, so they are written once and read once.  With dW their exponents are
// written (pack_exponents) and become dz = bf16 in place, which both products read.
// Either way a value is rounded to bf16 once, and is as exact beside a far likelier
// neighbour as alone.  A backward call from stored statistics multiplies the logits
// again and writes dz at once.
//
// All three products share one tile loop, bound by the matrix cores' power: 256
// values of the output's contiguous index (MFMA rows: a lane then holds eight
// neighbours of one output row, a 16-byte store) x 64 to 256 of its rows, 64 inner
// indices a step.  Accumulators stay in AGPRs, both tiles stream into LDS by DMA and
// operands are read half a step ahead.  Operands whose inner index is not contiguous
// (W in dh, both in dW) are transposed by the LDS reads themselves.  At V = 128256,
// D = 4096 the log-probabilities of 2048 rows take 1.59 to 1.67 ms (1290 to 1350 TF, by
// the card; torch's products of such sizes reach 1240 to 1390) and 4096 rows' loss and dh
// 6.6 to 6.8 ms, both products at 1270 to 1310 TF.
#include "head.h"

#include <cfloat>
#include <type_traits>

namespace qnf4 {
namespace {

constexpr int kThreads = 256;           // of the streaming kernels
constexpr int kStep = 64;               // inner indices per step
constexpr int kTileA = 256;             // values of the output's contiguous index
constexpr int kMaxSlots = 1024;         // partial tiles of dh
constexpr int kMaxSplits = 64;
constexpr float kLog2e = 1.4426950408889634f;

typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

constexpr float kLog2eLo = 1.925963033500e-08f;   // log2 e - kLog2e

// 2^t, t <= 0, kept in 16 bits: t as a whole number of steps of 90.5 / 65535, rounded to
// nearest, so 2^t is off by ln 2 / 2 steps, 2^-11 of itself, all the way down to 2^-90
// (63 nats); the last code is 0.  fp16 is as exact down to 2^-14 only and holds nothing
// below 2^-25: vocabulary entries 10 to 17 nats under the likeliest of their slice would
// lose their gradient, rows of dW that the norm of all does not show.  It costs what fp16
// does (2048 rows' loss, dh and dW at V = 128256, D = 4096: 5465 us, with fp16 5485).
// (A NaN leaves its whole row's factor NaN, whatever becomes of it here.)
constexpr float kExponents = 90.5f;
__device__ __forceinline__ uint32_t pack_exponents(float t, float u) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pknorm_u16(t * (-1.f / kExponents),
                                                                      u * (-1.f / kExponents)));
}
// 2^(by + t) of a code
__device__ __forceinline__ float unpack_power(uint32_t code, float by) {
  const float e = __builtin_fmaf((float)code, -kExponents / 65535.f, by);
  return code == 65535u ? 0.f : __builtin_amdgcn_exp2f(e);
}

__device__ __forceinline__ float exp_diff(float z, float m) {
  return __builtin_amdgcn_exp2f((z - m) * kLog2e);
}
// A slice's whole exponent for its largest logit m (finite also where m log2 e is not), and
// what 2^(z log2 e - M) has beside (z - m) log2 e: m log2 e - M, to float32's last bit
// while M is exact, and never out of [-1, 0] for logits beyond that (2^23).
__device__ __forceinline__ float slice_exponent(float m) {
  return fminf(fmaxf(ceilf(m * kLog2e), -FLT_MAX), FLT_MAX);
}
__device__ __forceinline__ float slice_offset(float m, float M) {
  return fminf(fmaxf(__builtin_fmaf(m, kLog2eLo, __builtin_fmaf(m, kLog2e, -M)), -1.f), 0.f);
}

// A slice's exponent relative to that of the row's largest logit, a whole number from -2000
// to 0.  (Where exponents are no longer exact their difference may be off by more than
// the logits': never above these.  -2000 too for a slice without entries or of NaN,
// whose sum shows it.)
__device__ __forceinline__ float relative_exponent(float slice, float row) {
  const float d = slice_exponent(slice) - slice_exponent(row);
  return fmaxf(fminf(d, ceilf((slice - row) * kLog2e) + 1.f), -2000.f);
}

// ----------------------------------------------------------------- slices of dh
// The inner index is the vocabulary, long: with fewer tiles than CUs it is cut
// into the number of slices that fills whole rounds best, which hangs on how
// many rows there are and so is found here.  A slice's epilogue and its part of
// the sum that follows cost about as much as 24 steps.
__host__ __device__ inline uint32_t dh_cost(uint32_t tiles, uint32_t steps, uint32_t splits) {
  const uint32_t each = (steps + splits - 1) / splits;
  if (splits > 1 && (each < 6 || tiles * splits > kMaxSlots)) return UINT32_MAX;
  return (tiles * splits + 255) / 256 * (each + (splits > 1 ? 24 : 4));
}
int dh_splits(int64_t tiles, int64_t steps) {
  if (tiles > kMaxSlots) return 1;
  int best = 1;
  for (int s = 2; s <= kMaxSplits; ++s)
    if (dh_cost(tiles, steps, s) < dh_cost(tiles, steps, best)) best = s;
  return best;
}
// the same by a wave, a candidate a lane
__device__ __forceinline__ int dh_splits_wave(int64_t tiles, int64_t steps, int lane) {
  if (tiles > kMaxSlots) return 1;
  uint64_t c = (uint64_t)dh_cost((uint32_t)tiles, (uint32_t)steps, lane + 1) << 8 | (lane + 1);
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const uint64_t o = __shfl_xor(c, d);
    c = o < c ? o : c;
  }
  return (int)(c & 255);
}

// ---------------------------------------------------------------- packing rows
// Bound by HBM where rows are many (3055 of 4096 rows at D = 4096: 27 us, 75 MB with the
// targets' rows of W, each of which a wave waits for), by latency below (5 us).
// Workgroup b looks after rows [b R, (b + 1) R): it counts the targets before
// them, copies its rows that have one to their places and clears what the call
// returns for the others.  Labels are few (8 bytes a row, against 2 D), so
// every workgroup counts for itself and one launch does.
__global__ __launch_bounds__(kThreads) void k_head_pack(HeadPackArgs a, int64_t per) {
  __shared__ int wave_count[4];
  __shared__ int place[kThreads];
  __shared__ double wave_sum[4];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t first = blockIdx.x * per;
  const int64_t end = first + per < a.rows ? first + per : a.rows;
  auto has = [&](int64_t t) { return a.labels[t] >= 0 && (!a.w || a.w[t] != 0.f); };
  int c = 0;
#pragma unroll 8
  for (int64_t t = tid; t < first; t += kThreads) c += has(t);
#pragma unroll
  for (int d = 32; d; d >>= 1) c += __shfl_xor(c, d);
  if (lane == 0) wave_count[wv] = c;
  __syncthreads();
  int at = wave_count[0] + wave_count[1] + wave_count[2] + wave_count[3];
  if (a.pad)
    for (int64_t v = (int64_t)blockIdx.x * kThreads + tid; v < a.vocab;
         v += (int64_t)gridDim.x * kThreads)
      a.to.last[v] = -1;
  const float scale = a.w && a.w_scale ? a.w_scale[0] : 1.f;
  const int chunks = a.dim / 8;
  // with one row a workgroup its four waves share the row's chunks
  const int ways = per == 1 ? 4 : 1, from = ways == 4 ? tid : lane, stride = 64 * ways;
  for (int64_t t0 = first; t0 < end; t0 += kThreads) {
    const int64_t t = t0 + tid;
    const bool mine = t < end && has(t);
    const uint64_t m = __builtin_amdgcn_ballot_w64(mine);
    __syncthreads();                       // the counts and places read before
    if (lane == 0) wave_count[wv] = __popcll(m);
    __syncthreads();
    int p = at + __popcll(m & ((1ull << lane) - 1));
    for (int w = 0; w < wv; ++w) p += wave_count[w];
    place[tid] = mine ? p : -1;
    if (mine) {
      const int64_t y = a.labels[t];
      a.to.src[p] = (int32_t)t;
      a.to.y[p] = y < a.vocab ? (int32_t)y : -1;
      if (a.w) {
        const float w = scale * a.w[t];
        a.to.w[p] = w;
        a.to.stat[p] = a.stat[t];
        a.to.scale[p] = HeadScale{0.f, 0.f, y < a.vocab ? w * a.stat[t].rest : NAN};
      }
    } else if (t < end) {
      if (a.logp) a.logp[t] = 0.f;
      if (a.stat_out) a.stat_out[t] = HeadStat{0.f, 0.f};
    }
    __syncthreads();
    const int n = end - t0 < kThreads ? (int)(end - t0) : kThreads;
    for (int i = ways == 4 ? 0 : wv; i < n; i += 4 / ways) {
      const int q = place[i];
      const uint4* in = reinterpret_cast<const uint4*>(a.hidden + (t0 + i) * a.ldh);
      if (q >= 0) {
        uint4* out = reinterpret_cast<uint4*>(a.to.h + (int64_t)q * a.dim);
        const int64_t y = a.labels[t0 + i];
        if (!a.weight || y >= a.vocab) {
#pragma unroll 4
          for (int k = from; k < chunks; k += stride) out[k] = in[k];
          continue;
        }
        // the target's logit, in float64: logp and 1 - p of a likely target hang on its
        // last bits (from the product's float32 sum logp of one row at D = 4096 was
        // off by 6e-6 of itself, and torch's by 5e-7)
        const uint4* with = reinterpret_cast<const uint4*>(a.weight + y * a.ldw);
        double z = 0;
#pragma unroll 4
        for (int k = from; k < chunks; k += stride) {
          const uint4 x = in[k], w = with[k];
          out[k] = x;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t u = (&x.x)[e], v = (&w.x)[e];
            z += (double)(bf16_to_f32((uint16_t)u) * bf16_to_f32((uint16_t)v)) +
                 (double)(bf16_to_f32((uint16_t)(u >> 16)) * bf16_to_f32((uint16_t)(v >> 16)));
          }
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) z += __shfl_xor(z, d);
        if (ways == 4) {
          if (lane == 0) wave_sum[wv] = z;
          __syncthreads();
          z = wave_sum[0] + wave_sum[1] + wave_sum[2] + wave_sum[3];
        }
        if (lane == 0 && (ways == 1 || wv == 0)) a.to.zy[q] = z;
      } else if (a.dh) {
        uint4* out = reinterpret_cast<uint4*>(a.dh + (t0 + i) * a.ldd);
        for (int k = from; k < chunks; k += stride) out[k] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    at += wave_count[0] + wave_count[1] + wave_count[2] + wave_count[3];
  }
  if (blockIdx.x != gridDim.x - 1) return;
  // how many, and the slices of dh over a last panel that they do not fill
  if (wv == 0) {
    const int rest = at % a.panel;
    const int sp = dh_splits_wave(ceil_div(a.dim, kTileA) * ceil_div(rest, a.tile),
                                  ceil_div(a.vocab, kStep), lane);
    if (lane == 0) {
      a.to.n[0] = at;
      a.to.n[1] = sp;
    }
  }
  if (!a.pad) return;
  // zeros up to a whole step: inner indices of dW
  for (int64_t q = at + wv; q < ceil_div(at, kStep) * kStep; q += 4) {
    uint4* out = reinterpret_cast<uint4*>(a.to.h + q * a.dim);
    for (int k = lane; k < chunks; k += 64) out[k] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// ----------------------------------------------------------------- tile loop
__device__ __forceinline__ void mfma_acc(f32x4_t& acc, const u32x4_t& a, const u32x4_t& b) {
  // (results in AGPRs by hand: with 256 of them in use the allocator otherwise
  // moves tiles to VGPRs and back every step)
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma_settle() { asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7"); }

// f(I), ..., f(N - 1) with constants (the unroller gives up on the step's body)
template <int I, int N, typename F>
__device__ __forceinline__ void static_for(const F& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<I + 1, N>(f);
  }
}

constexpr int min_of(int a, int b) { return a < b ? a : b; }

template <int N>
__device__ __forceinline__ void wait_vmem() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// 16 bytes a lane from base + off to LDS address lds + 16 lane (as dma16, with the
// lane's part of the address in 32 bits)
__device__ __forceinline__ void dma16_at(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(off), "s"(base), "s"(lds) : "m0", "memory");
}

__device__ __forceinline__ void dma4_at(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :: "v"(off), "s"(base), "s"(lds) : "m0", "memory");
}

// An operand: element (index, inner) at p[index * ld + inner] (TR false) or
// p[inner * ld + index] (TR true); indices past `count` repeat the last ones
// (their outputs are not stored), inner indices past `inner` the last one (the
// other operand is zero there).  TR: count % 8 == 0.
struct Operand {
  const uint16_t* p;
  int64_t ld;
  int64_t count, inner;
};

// LDS of a step.  TR false: [R][64] values, 128 bytes a row, 16-byte chunk c of row
// r at c ^ hash(r); TR true: [64][R], 2 R bytes an inner index k, chunk c at
// c ^ hash(k).  The hashes spread what the lanes of a read use together over all 64
// banks: A's MFMA row 4 q + v of tile (i, h) is index 32 i + 8 q + 4 h + v (so that
// a lane's results of h = 0, 1 are neighbours), B's is in order.
template <int R, bool TR, bool IS_A, int WAVES>
struct Tile {
  static constexpr int kBytes = R * kStep * 2;
  static constexpr int kLoads = kBytes / 1024 / WAVES;     // per wave and step
  static constexpr int kRowChunks = TR ? R / 8 : 8;
  uint32_t off[kLoads];
  uint32_t krow[TR ? kLoads : 1];
  const uint16_t* base;
  uint32_t ld2;
  int64_t inner;

  __device__ static __forceinline__ int hash(int r) {
    if (TR) return (IS_A ? (r & 1) | ((r & 2) << 1) : (r & 3) << 1) | (r & 8);
    return IS_A ? (r & 3) | (((r >> 3) & 1) << 2) : r & 7;
  }
  __device__ __forceinline__ void init(const Operand& o, int64_t first, int lane, int wv) {
    ld2 = (uint32_t)(o.ld * 2);
    inner = o.inner;
    base = TR ? o.p + first : o.p + first * o.ld;
    const int64_t left = o.count - first;      // > 0
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int chunk = (kLoads * wv + q) * 64 + lane;
      const int row = chunk / kRowChunks;
      const int c = (chunk % kRowChunks) ^ hash(row);
      if (TR) {
        krow[q] = row;
        const int64_t col = 8 * c < left ? 8 * c : left - 8;
        off[q] = (uint32_t)(col * 2);
      } else {
        const int64_t r = row < left ? row : left - 1;
        off[q] = (uint32_t)r * ld2 + 16 * c;
      }
    }
  }
  // load q of step k0 / 64
  __device__ __forceinline__ void load(int q, int64_t k0, uint32_t lds, int wv) const {
    const uint32_t to = lds + (kLoads * wv + q) * 1024;
    if (TR) {
      const int64_t left = inner - 1 - k0;
      const uint32_t k = (int64_t)krow[q] < left ? krow[q] : (uint32_t)left;
      dma16_at(base + k0 * (ld2 / 2), off[q] + __umul24(k, ld2), to);
    } else {
      dma16_at(base + k0, off[q], to);
    }
  }
  // A lane's addresses within a stage: kBases of them, a tile's at one of them (plus a
  // constant where the tile's bits are none that the hash reaches).
  static constexpr int kBases = TR ? 8 : 2;
  __device__ static __forceinline__ void bases(uint32_t (&b)[kBases], int first, int lane) {
    const int j = lane & 15, g = lane >> 4;
    if (!TR) {
      const int row = IS_A ? 8 * (j >> 2) + (j & 3) : j;
#pragma unroll
      for (int s = 0; s < 2; ++s)
        b[s] = (first + row) * 128 + (((4 * s + g) ^ hash(row)) << 4);
    } else {
      // this lane hands in 8 bytes of inner index 8 g + j / 4, piece j % 4 of 16 columns
      const int k = 8 * g + (j >> 2), p = j & 3;
#pragma unroll
      for (int t = 0; t < kBases; ++t) {
        const int c = IS_A ? 4 * (t >> 1) + p : 2 * t + (p >> 1);
        const int half = IS_A ? (t & 1) ^ (p & 1) : p & 1;
        b[t] = k * R * 2 + (((first / 8 + c) ^ hash(k)) << 4) + 8 * half;
      }
    }
  }
  // MFMA operand of tile t (A: t = 2 i + h), half s of the step
  __device__ static __forceinline__ u32x4_t read(const char* lds, const uint32_t (&b)[kBases],
                                                 int t, int s) {
    if constexpr (!TR) {
      const int c = IS_A ? (t >> 1) * 4096 + (t & 1) * 512 : t * 2048;
      return *reinterpret_cast<const u32x4_t*>(lds + b[s] + c);
    } else {
      const char* at = lds + b[t] + s * 32 * R * 2;
      const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)at);
      const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(at + 4 * R * 2));
      const uint2 l = __builtin_bit_cast(uint2, lo), u = __builtin_bit_cast(uint2, hi);
      return u32x4_t{l.x, l.y, u.x, u.y};
    }
  }
};

// Exponents that a B operand's bf16 values are lowered by before they are multiplied:
// rows' words (the same in both halves) p[(inner / 128) * ld + row].
struct Shift {
  const uint32_t* p;
  int64_t ld;
};

// TN rows of B, WB waves along them (and two along A).
template <int TN, int WB, bool SHIFT = false>
struct Shape {
  static constexpr int kWaves = 2 * WB;
  static constexpr int kTilesB = TN / 16 / WB;     // MFMA tiles of a wave
  // 256 rows: A in three buffers and B in two fill LDS (the words of SHIFT leave A two)
  static constexpr bool kA3 = TN == 256 && !SHIFT;
  static constexpr int kStages = TN == 256 ? 2 : 3;        // of B
  static constexpr int kStagesA = kA3 ? 3 : kStages;
  static constexpr int kA = kTileA * kStep * 2, kB = TN * kStep * 2, kWords = SHIFT ? TN * 4 : 0;
  // a step's A, B and words side by side, or A's buffers and then B's
  static constexpr int kStage = kA + kB + kWords;
  static constexpr uint32_t kNextA = kA3 ? kA : kStage, kNextB = kA3 ? kB : kStage;
  static constexpr uint32_t kEndA = kStagesA * kNextA, kEndB = kStages * kNextB;
  static constexpr int kAtB = kA3 ? kEndA : kA, kAtWords = kAtB + kB;
  static constexpr int kLds = kA3 ? kEndA + kEndB : kEndB;
};

// acc[ta][tb] += A . B^T over steps [s0, s1) (s0 < s1).  Wave (wm, wn): A's values
// 128 wm .. and B's rows TN / WB wn ...  While a half step is multiplied from
// registers, the next half's operands are read.  One barrier a step, in its
// middle: by then every wave has read the step's second half, so its buffers are
// free, and step k + 1's tiles have landed (an exact vmcnt: every wave issues the
// same loads each step, past the end the last step's again).
//
// The loads' path takes 64 bytes a cycle, half of a step's time at 256 rows, and what
// comes faster holds up the wave: bunched in a quarter of the step the products ran
// 7% slower than over half of it.  So A has a third buffer where LDS has room: its
// tile of step k + 2 goes there in the first half of step k, B's in the second
// half, to the buffer that step k leaves (V = 128256, D = 4096: 2048 rows' loss, dh and
// dW 5550 -> 5385 us; logits of 2048 rows at V = 32000, D = 8192: 849 -> 825).
template <int TN, int WB, bool ATR, bool BTR, bool SHIFT = false>
__device__ __forceinline__ void tile_loop(f32x4_t (&acc)[8][TN / 16 / WB], char* lds,
                                          const Operand& A, int64_t a0, const Operand& B,
                                          int64_t b0, int64_t s0, int64_t s1,
                                          const Shift& sh = Shift{nullptr, 0}) {
  using S = Shape<TN, WB, SHIFT>;
  using TA = Tile<kTileA, ATR, true, S::kWaves>;
  using TB = Tile<TN, BTR, false, S::kWaves>;
  constexpr int NB = S::kTilesB, NS = S::kStages;
  constexpr int LA = TA::kLoads, LB = TB::kLoads + SHIFT;
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv & 1, wn = wv >> 1;
  TA ta;
  TB tb;
  ta.init(A, a0, lane, wv);
  tb.init(B, b0, lane, wv);
  uint32_t ab[TA::kBases], bb[TB::kBases];
  TA::bases(ab, 128 * wm, lane);
  TB::bases(bb, 16 * NB * wn, lane);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void_t*)lds;

#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int t = 0; t < NB; ++t) {
      acc[i][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      asm volatile("" : "+a"(acc[i][t]));
    }
  mfma_settle();

  // buffers by where they are behind the first: A's, B's (and its words')
  auto inner = [&](int64_t step) __attribute__((always_inline)) {
    return (step < s1 ? step : s1 - 1) * kStep;
  };
  auto load_a = [&](int q, int64_t step, uint32_t buf) __attribute__((always_inline)) {
    ta.load(q, inner(step), lds0 + buf, wv);
  };
  auto load_b = [&](int q, int64_t step, uint32_t buf) __attribute__((always_inline)) {
    if (q < TB::kLoads) tb.load(q, inner(step), lds0 + S::kAtB + buf, wv);
    else   // (several waves fetch the same words where there are more waves than those)
      dma4_at(sh.p + inner(step) / 128 * sh.ld + b0 + 64 * (wv % (TN / 64)), 4 * lane,
              lds0 + S::kAtWords + buf + 256 * (wv % (TN / 64)));
  };
#pragma unroll
  for (int st = 0; st < NS; ++st) {
#pragma unroll
    for (int q = 0; q < LA; ++q) load_a(q, s0 + st, st * S::kNextA);
#pragma unroll
    for (int q = 0; q < LB; ++q) load_b(q, s0 + st, st * S::kNextB);
  }
  wait_vmem<(NS - 1) * (LA + LB)>();
  __syncthreads();

  u32x4_t fa[2][8], fb[2][NB];
  // operand r of half s
  auto fetch = [&](int r, uint32_t ba, uint32_t bb0, int s) __attribute__((always_inline)) {
    if (r < 8) fa[s][r] = TA::read(lds + ba, ab, r, s);
    else fb[s][r - 8] = TB::read(lds + S::kAtB + bb0, bb, r - 8, s);
  };
#pragma unroll
  for (int r = 0; r < 8 + NB; ++r) fetch(r, 0, 0, 0);

  // The exponents of bf16 values by whole numbers: exact, and 0 where one would leave the
  // range.  A tile's words are changed at least two instructions before the first
  // product that reads them (which the compiler does not see inside the asm).
  uint32_t sv[NB];
  auto words = [&](int t, uint32_t buf) __attribute__((always_inline)) {
    if constexpr (SHIFT)
      sv[t] = *reinterpret_cast<const uint32_t*>(lds + S::kAtWords + buf +
                                                 4 * (16 * (NB * wn + t) + (lane & 15)));
  };
  auto lower = [&](int t, int s) __attribute__((always_inline)) {
    if constexpr (SHIFT) {
      const u16x2_t by = __builtin_bit_cast(u16x2_t, sv[t]);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        fb[s][t][q] = __builtin_bit_cast(
            uint32_t, __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2_t, (uint32_t)fb[s][t][q]), by));
    }
  };
#pragma unroll
  for (int t = 0; t < NB; ++t) words(t, 0);
  lower(0, 0);

  constexpr int M = 8 * NB, R = 8 + NB, RM = M * 3 / 4;
  // loads of the second half: B's, and A's where it has no buffer of its own
  constexpr int L1 = S::kA3 ? LB : LA + LB;
  uint32_t ca = 0, cb3 = 0;                       // this step's buffers
  for (int64_t k = s0; k < s1; ++k) {
    const uint32_t cb = S::kA3 ? cb3 : ca;
    auto after = [](uint32_t at, uint32_t next, uint32_t end) __attribute__((always_inline)) {
      return at + next == end ? 0u : at + next;
    };
    const uint32_t na = after(ca, S::kNextA, S::kEndA);
    const uint32_t nb = S::kA3 ? after(cb, S::kNextB, S::kEndB) : na;
    const uint32_t free_a = S::kA3 ? after(na, S::kNextA, S::kEndA) : ca;
    if constexpr (SHIFT) asm volatile("s_nop 1");
    static_for<0, M>([&](auto c) __attribute__((always_inline)) {
      constexpr int i = c;
      mfma_acc(acc[i & 7][i >> 3], fa[0][i & 7], fb[0][i >> 3]);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (S::kA3)
        static_for<i * LA / M, (i + 1) * LA / M>(
            [&](auto q) __attribute__((always_inline)) { load_a(q, k + 2, free_a); });
      static_for<min_of(i * R / RM, R), min_of((i + 1) * R / RM, R)>(
          [&](auto r) __attribute__((always_inline)) { fetch(r, ca, cb, 1); });
      if constexpr (i % 8 == 4 && i / 8 + 1 < NB) lower(i / 8 + 1, 0);
      if constexpr (i == M - 1) lower(0, 1);
      __builtin_amdgcn_sched_barrier(0);
    });
    wait_vmem<S::kA3 ? LA : (NS - 2) * (LA + LB)>();
    __syncthreads();
    static_for<0, M>([&](auto c) __attribute__((always_inline)) {
      constexpr int i = c;
      mfma_acc(acc[i & 7][i >> 3], fa[1][i & 7], fb[1][i >> 3]);
      __builtin_amdgcn_sched_barrier(0);
      static_for<i * L1 / M, (i + 1) * L1 / M>([&](auto q) __attribute__((always_inline)) {
        if constexpr (q < L1 - LB) load_a(q, k + NS, free_a);
        else load_b(q - (L1 - LB), k + NS, cb);
      });
      static_for<min_of(i * R / RM, R), min_of((i + 1) * R / RM, R)>(
          [&](auto r) __attribute__((always_inline)) { fetch(r, na, nb, 0); });
      if constexpr (i % 8 == 4 && i / 8 + 1 < NB) lower(i / 8 + 1, 1);
      // (the last tile's words are used by then)
      if constexpr (i >= RM && i < RM + NB) words(i - RM, nb);
      if constexpr (i == M - 1) lower(0, 0);
      __builtin_amdgcn_sched_barrier(0);
    });
    ca = na;
    cb3 = nb;
  }
  wait_vmem<0>();   // nothing left in flight into LDS at exit
  mfma_settle();
}

// Tile of workgroup `id` among na x nb (A tiles, B tiles): workgroups go to the
// eight XCDs in turn, so each XCD takes a contiguous run of the order "eight A
// tiles, then the next B tile", where 32 neighbours (its CUs) share 8 + 4 tiles.
// With slices of the inner index, all tiles of one, then the next.
__device__ __forceinline__ bool tile_of(int64_t id, int64_t na, int64_t nb, int64_t& ta,
                                        int64_t& tb, int slices = 1, int* slice = nullptr) {
  const int64_t tiles = na * nb, total = tiles * slices, per = ceil_div(total, 8);
  const int64_t loc = id >> 3;
  int64_t l = (id & 7) * per + loc;
  if (loc >= per || l >= total) return false;
  if (slice) {
    *slice = (int)(l / tiles);
    l -= *slice * tiles;
  }
  const int64_t grp = l / (8 * nb), left = na - 8 * grp;
  const int64_t rem = l - grp * 8 * nb, ga = left < 8 ? left : 8;
  tb = rem / ga;
  ta = 8 * grp + rem % ga;
  return true;
}

__device__ __forceinline__ int panel_rows(const HeadPanel& p) {
  const int64_t n = __builtin_amdgcn_readfirstlane(*p.r.n) - p.row0;
  return n < 0 ? 0 : n < p.rows ? (int)n : p.rows;
}

__device__ __forceinline__ int panel_splits(const HeadPanel& p, int n) {
  return n == p.rows ? p.splits : __builtin_amdgcn_readfirstlane(p.r.n[1]);
}

// -------------------------------------------------------------------- logits
// A = W (the vocabulary along a lane's registers: a row's statistics are sums in the
// lane, then over the four lanes of its column), B = rows.  One row of 4096 reads a
// weight of 128256 rows in 171 us, 6.1 TB/s; many rows are bound by the matrix cores.
constexpr int HEAD_RAW = 4;    // partial logits of a slice of the inner index
// Waves along the rows.  Of 256 rows, two of 128 each read half as much from LDS as
// four of 64 do, for one wave a SIMD: 2048 rows at D = 8192, V = 32000 take 813 us for
// 825.  Where powers for dh are written the wave's epilogue costs more than that (4096
// rows at V = 128256, D = 4096, loss and dh: 6835 us for 6789), and the products that
// transpose lose as well (2048 rows' loss, dh and dW: 5650 with two waves in dh and
// 5861 with two in dW, for 5561).
constexpr int kWavesB = 4;
constexpr int logits_waves(int tn, int mode) {
  return tn == 256 && mode != HEAD_POW ? 2 : kWavesB;
}
template <int TN, int MODE, int WB>
__global__ __attribute__((amdgpu_flat_work_group_size(128 * WB, 128 * WB),
                          amdgpu_waves_per_eu(WB / 2, WB / 2)))
void k_head_logits(HeadPanel p, int splits, float* part) {
  __shared__ __attribute__((aligned(1024))) char lds[Shape<TN, WB>::kLds];
  constexpr int NB = Shape<TN, WB>::kTilesB;
  const int n = panel_rows(p);
  const int64_t na = ceil_div(p.vocab, kTileA), nb = ceil_div(n, TN);
  int64_t tv, tt;
  int sl;
  if (!tile_of(blockIdx.x, na, nb, tv, tt, MODE == HEAD_RAW ? splits : 1, &sl)) return;
  const int64_t steps = p.dim / kStep, each = MODE == HEAD_RAW ? ceil_div(steps, splits) : steps;
  const Operand A{p.weight, p.ldw, p.vocab, p.dim};
  const Operand B{p.r.h + p.row0 * p.dim, p.dim, n, p.dim};
  f32x4_t acc[8][NB];
  // (no slice is empty: logits_splits)
  tile_loop<TN, WB, false, false>(acc, lds, A, tv * kTileA, B, tt * TN, sl * each,
                                  (sl + 1) * each < steps ? (sl + 1) * each : steps);

  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv & 1, wn = wv >> 1;
  const int64_t v0 = tv * kTileA + 128 * wm;       // of this wave's slice
  const int64_t cols = head_cols(p.vocab);
#pragma unroll
  for (int t = 0; t < NB; ++t) {
    const int row = (int)(tt * TN) + 16 * (NB * wn + t) + j;
    const bool valid = row < n;
    if constexpr (MODE == HEAD_RAW) {
      float* to = part + ((sl * na + tv) * nb + tt) * (TN * kTileA) +
                  (row - tt * TN) * kTileA + 128 * wm + 8 * g;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<f32x4_t*>(to + 32 * (i >> 1) + 4 * (i & 1)) = acc[i][t];
      continue;
    }
    const int64_t q = p.row0 + (valid ? row : 0);
    const int64_t rel = valid ? (int64_t)p.r.y[q] - v0 - 8 * g : -1;   // in this lane: 32 i + 4 h + v
    float z[32];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) z[4 * i + v] = acc[i][t][v];
    if (v0 + 128 > p.vocab) {   // the vocabulary's last tile
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (v0 + 32 * (i >> 3) + 8 * g + (i & 7) >= p.vocab) z[i] = -INFINITY;
    }
    uint16_t* out = p.e + (int64_t)row * cols + v0 + 8 * g;
    if (MODE == HEAD_DZ) {
      const HeadStat st = p.r.stat[q];
      const float w = p.r.w[q];
#pragma unroll
      for (int i = 0; i < 32; ++i) z[i] = -w * exp_diff(z[i], st.lse);
      if (__builtin_amdgcn_ballot_w64(rel >= 0 && rel < 128)) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (rel == 32 * (i >> 3) + (i & 7)) {
            z[i] = w * st.rest;
            if (p.want_last) atomicMax(p.r.last + p.r.y[q], (int)q);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 o = make_uint4(pack_bf16x2(z[8 * i], z[8 * i + 1]),
                             pack_bf16x2(z[8 * i + 2], z[8 * i + 3]),
                             pack_bf16x2(z[8 * i + 4], z[8 * i + 5]),
                             pack_bf16x2(z[8 * i + 6], z[8 * i + 7]));
        // (rows behind the last are inner indices of dW, whatever h holds there)
        if (!valid) o = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(out + 32 * i) = o;
      }
      continue;
    }
    if (__builtin_amdgcn_ballot_w64(rel >= 0 && rel < 128)) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (rel == 32 * (i >> 3) + (i & 7)) {
          z[i] = -INFINITY;
          if (MODE == HEAD_EXP) atomicMax(p.r.last + p.r.y[q], (int)q);
        }
    }
    float m = z[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) m = fmaxf(m, z[i]);
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    const float M = slice_exponent(m), off = slice_offset(m, M), from = m == -INFINITY ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float t = __builtin_fmaf(z[i] - from, kLog2e, off), e = __builtin_amdgcn_exp2f(t);
      z[i] = MODE == HEAD_EXP ? t : e;
      s += e;
    }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (valid && g == 0) p.part[(2 * tv + wm) * p.rows + row] = HeadPart{m, s};
    if ((MODE == HEAD_EXP || MODE == HEAD_POW) && valid) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          o[k] = MODE == HEAD_POW
                     ? pack_bf16x2(z[8 * i + 2 * k], z[8 * i + 2 * k + 1])
                     : pack_exponents(z[8 * i + 2 * k], z[8 * i + 2 * k + 1]);
        *reinterpret_cast<uint4*>(out + 32 * i) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// With few tiles (a small vocabulary, few rows) the logits' inner index is cut over
// the CUs and this kernel adds the parts and does what the tile's epilogue does
// otherwise: a wave per row and slice of 128 vocabulary entries, two a lane.
template <int MODE>
__global__ __launch_bounds__(kThreads) void k_head_slices(HeadPanel p, int TN, int splits,
                                                          const float* part) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int n = panel_rows(p);
  const int row = blockIdx.x * 4 + wv, sl = blockIdx.y;
  // (rows behind the last: zeros for dW's inner index)
  const int rows = MODE == HEAD_DZ ? (int)ceil_div(n, kStep) * kStep : n;
  if (row >= rows) return;
  const int64_t na = ceil_div(p.vocab, kTileA), nb = ceil_div(n, TN), cols = head_cols(p.vocab);
  const int64_t v = 128 * (int64_t)sl + 2 * lane;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.e + row * cols + v);
  if (MODE == HEAD_DZ && row >= n) {
    *out = 0u;
    return;
  }
  const float* from = part + ((sl >> 1) * nb + row / TN) * (TN * kTileA) + (row % TN) * kTileA +
                      128 * (sl & 1) + 2 * lane;
  float z[2] = {0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float2 x = *reinterpret_cast<const float2*>(from + s * (na * nb * (TN * kTileA)));
    z[0] += x.x;
    z[1] += x.y;
  }
  const int64_t q = p.row0 + row;
  const int y = p.r.y[q];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (v + e >= p.vocab) z[e] = -INFINITY;
  if (MODE == HEAD_DZ) {
    const HeadStat st = p.r.stat[q];
    const float w = p.r.w[q];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      z[e] = -w * exp_diff(z[e], st.lse);
      if (v + e == y) {
        z[e] = w * st.rest;
        if (p.want_last) atomicMax(p.r.last + y, (int)q);
      }
    }
    *out = pack_bf16x2(z[0], z[1]);
    return;
  }
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (v + e == y) {
      z[e] = -INFINITY;
      if (MODE == HEAD_EXP) atomicMax(p.r.last + y, (int)q);
    }
  float m = fmaxf(z[0], z[1]);
#pragma unroll
  for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float M = slice_exponent(m), off = slice_offset(m, M), at = m == -INFINITY ? 0.f : m;
  float t[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    t[e] = __builtin_fmaf(z[e] - at, kLog2e, off);
    z[e] = __builtin_amdgcn_exp2f(t[e]);
  }
  float s = z[0] + z[1];
#pragma unroll
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  if (lane == 0) p.part[(int64_t)sl * p.rows + row] = HeadPart{m, s};
  if (MODE == HEAD_POW) *out = pack_bf16x2(z[0], z[1]);
  if (MODE == HEAD_EXP) *out = pack_exponents(t[0], t[1]);
}

// ---------------------------------------------------------------------- join
// A workgroup joins the slices of 16 rows, 64 of its threads a row: the maximum
// first, then the sums in float64.  Latency: 5 us for 250 slices a row, 11 for 1002
// (16 loads in flight a thread, kept for the second pass).
constexpr int kJoinRows = 16, kJoinWaves = 16;
__global__ __launch_bounds__(64 * kJoinWaves)
void k_head_join(HeadPanel p, int kind, int shift, double* lp, float* logp, HeadStat* stat) {
  __shared__ float ms[kJoinWaves][kJoinRows];
  __shared__ double ss[kJoinWaves][kJoinRows];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, r = lane & 15;
  const int n = panel_rows(p);
  const int row = blockIdx.x * kJoinRows + r;
  if ((int)blockIdx.x * kJoinRows >= n) return;
  const int rr = row < n ? row : n - 1;
  const int64_t slices = 2 * ceil_div(p.vocab, kTileA);
  const HeadPart* part = p.part + rr;
  const int first = 4 * wv + (lane >> 4);
  // (a thread's first 16 slices stay in registers: a vocabulary of 131072)
  constexpr int kHeld = 16, kStride = 4 * kJoinWaves;
  HeadPart held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int64_t sl = first + k * kStride;
    held[k] = sl < slices ? part[sl * p.rows] : HeadPart{-INFINITY, 0.f};
  }
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) m = fmaxf(m, held[k].m);
#pragma unroll 8
  for (int64_t k = first + kHeld * kStride; k < slices; k += kStride)
    m = fmaxf(m, part[k * p.rows].m);
  m = fmaxf(m, __shfl_xor(m, 16));
  m = fmaxf(m, __shfl_xor(m, 32));
  if (lane < 16) ms[wv][r] = m;
  const int32_t y = p.r.y[p.row0 + rr];
  const double zy = y >= 0 ? p.r.zy[p.row0 + rr] : NAN;
  __syncthreads();
  m = ms[0][r];
#pragma unroll
  for (int k = 1; k < kJoinWaves; ++k) m = fmaxf(m, ms[k][r]);
  // sums relative to 2^M of the row: every factor is a power of two
  double s = 0;
  auto add = [&](const HeadPart& e, int64_t k) {
    const int down = (int)relative_exponent(e.m, m);
    s += ldexp((double)e.s, down);
    if (shift && row < n) {
      const uint32_t d = down < -511 ? 511 : -down;
      p.shift[k * p.rows + row] = e.s == 0.f ? 0u : d << 7 | d << 23;
    }
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (first + k * kStride < slices) add(held[k], first + k * kStride);
#pragma unroll 8
  for (int64_t k = first + kHeld * kStride; k < slices; k += kStride) add(part[k * p.rows], k);
  s += __shfl_xor(s, 16);
  s += __shfl_xor(s, 32);
  if (lane < 16) ss[wv][r] = s;
  __syncthreads();
  if (threadIdx.x >= kJoinRows || row >= n) return;
  s = 0;
#pragma unroll
  for (int k = 0; k < kJoinWaves; ++k) s += ss[k][r];
  // the target joins: both relative to the larger logit's exponential.  (From that logit
  // itself, not from its exponent: lse of a far larger one is that float32, and the
  // backward's exp(z - lse) is 1 there.)
  const double top = fmax((double)m, zy);
  const float off = slice_offset(m, slice_exponent(m));
  const double out = m == -INFINITY ? 0.0 : exp((double)m - top) * exp2(-(double)off);
  const double rest = m == -INFINITY ? 0.0 : s * out, all = rest + exp(zy - top);
  const double lse = top + log(all);
  double l = zy - lse;
  HeadStat st{(float)lse, (float)(rest / all)};
  const double w = kind == HEAD_GRAD_MEAN ? -1.0 / *p.r.n : -1.0;
  HeadScale sc{m, (float)(-w * out / all), (float)(w * rest / all)};
  if (y < 0) {
    l = NAN;
    st = HeadStat{NAN, NAN};
    sc = HeadScale{0.f, NAN, NAN};
  }
  const int64_t q = p.row0 + row;
  const int32_t src = p.r.src[q];
  if (logp) logp[src] = (float)l;
  if (stat) stat[src] = st;
  if (kind >= HEAD_LOSS) lp[q] = l;
  if (kind >= HEAD_GRAD_SUM) p.r.scale[q] = sc;
}

// loss = -(sum of logp), over the number of targets
__global__ __launch_bounds__(1024) void k_head_loss(const int32_t* n, const double* lp, int mean,
                                                    float* loss) {
  __shared__ double ss[16];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, rows = *n;
  double s = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < rows; i += 1024) s += lp[i];
#pragma unroll
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  if (lane == 0) ss[wv] = s;
  __syncthreads();
  if (threadIdx.x) return;
  s = 0;
  for (int k = 0; k < 16; ++k) s += ss[k];
  *loss = (float)(rows == 0 ? 0.0 : mean ? -s / rows : -s);
}

// ------------------------------------------------------------------------ dz
// In place, a thread 8 columns of 8 rows: HBM-bound (2048 x 128256: 192 us, 1.05 GB at
// 5.5 TB/s).  dz = f 2^(M - R + t), the target's c; zeros in the rows up to a whole step of
// dW.
constexpr int kDzRows = 8;
__global__ __launch_bounds__(kThreads) void k_head_dz(HeadPanel p) {
  const int n = panel_rows(p);
  const int64_t cols = head_cols(p.vocab);
  const int64_t c = (int64_t)blockIdx.y * kThreads * 8 + threadIdx.x * 8;
  const int r0 = blockIdx.x * kDzRows;
  if (c >= cols || r0 >= (int)ceil_div(n, kStep) * kStep) return;
  uint4 e[kDzRows];
  uint4* at = reinterpret_cast<uint4*>(p.e + (int64_t)r0 * cols + c);
#pragma unroll
  for (int r = 0; r < kDzRows; ++r)
    e[r] = r0 + r < n ? at[r * (cols / 8)] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int r = 0; r < kDzRows; ++r) {
    uint4 o = make_uint4(0u, 0u, 0u, 0u);
    if (r0 + r < n) {
      const int64_t q = p.row0 + r0 + r;
      const HeadScale sc = p.r.scale[q];
      const float m = p.part[(c >> 7) * p.rows + r0 + r].m;
      const float by = relative_exponent(m, sc.m);
      float d[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t two = (&e[r].x)[k];
        d[2 * k] = sc.f * unpack_power(two & 0xffffu, by);
        d[2 * k + 1] = sc.f * unpack_power(two >> 16, by);
      }
      const int64_t rel = p.r.y[q] - c;
      if (rel >= 0 && rel < 8) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (rel == k) d[k] = sc.c;
      }
      o = make_uint4(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]), pack_bf16x2(d[4], d[5]),
                     pack_bf16x2(d[6], d[7]));
    }
    at[r * (cols / 8)] = o;
  }
}

// ------------------------------------------------------------------------ dh
// Eight neighbouring values of a lane: tiles (i, 0) and (i, 1), in the order the
// transposing read has them (odd lane groups the other way round).
template <int NB>
__device__ __forceinline__ void eight(const f32x4_t (&acc)[8][NB], int i, int t, int g,
                                      float (&o)[8]) {
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const float a = acc[2 * i][t][v], b = acc[2 * i + 1][t][v];
    o[v] = (g & 1) ? b : a;
    o[4 + v] = (g & 1) ? a : b;
  }
}
__device__ __forceinline__ uint4 pack8(const float (&o)[8]) {
  return make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                    pack_bf16x2(o[6], o[7]));
}

// A = W (transposed by the reads), B = e; inner index the vocabulary.  2048 rows at
// V = 128256, D = 4096 1.5 ms, 1400 TF, from dz; from powers, whose exponents the
// loop lowers on the vector unit, 3055 rows 2.6 ms, 1230 TF (192 tiles: cut in slices).
// POW: e holds 2^(z log2 e - M) of each slice: the tile loop lowers its exponents to
// the row's R, and what is left is a factor of the whole row and the target's term,
// c times its row of W, in float32 at the end.  So dz is rounded to bf16 once, e is
// written once and read once, and the target's cancellation stays out of the sums.
// From dz, the target's own rounding is put right the same way: it is the largest
// of its row, half of the gradient's error (2.4e-3 of its norm against 1.7e-3).
__device__ __forceinline__ void finish_row(const HeadPanel& p, bool pow, int64_t q, int64_t col,
                                           float (&o)[8]) {
  const HeadScale sc = p.r.scale[q];
  const int y = p.r.y[q];
  const uint4 w = *reinterpret_cast<const uint4*>(p.weight + (y < 0 ? 0 : y) * p.ldw + col);
  const float f = pow ? sc.f : 1.f;
  const float c = pow ? sc.c : sc.c - bf16_to_f32((uint16_t)pack_bf16x2(sc.c, 0.f));
#pragma unroll
  for (int k = 0; k < 8; ++k)
    o[k] = f * o[k] + c * bf16_to_f32((uint16_t)((&w.x)[k >> 1] >> (16 * (k & 1))));
}

template <int TN, bool POW>
__global__ __attribute__((amdgpu_flat_work_group_size(128 * kWavesB, 128 * kWavesB),
                          amdgpu_waves_per_eu(kWavesB / 2, kWavesB / 2)))
void k_head_dh(HeadPanel p, float* part, uint16_t* dh, int64_t ldd) {
  __shared__ __attribute__((aligned(1024))) char lds[Shape<TN, kWavesB, POW>::kLds];
  constexpr int NB = Shape<TN, kWavesB>::kTilesB;
  const int n = panel_rows(p), splits = panel_splits(p, n);
  const int64_t na = ceil_div(p.dim, kTileA), nb = ceil_div(n, TN);
  int64_t td, tt;
  int sl;
  if (!tile_of(blockIdx.x, na, nb, td, tt, splits, &sl)) return;
  const int64_t steps = ceil_div(p.vocab, kStep), each = ceil_div(steps, splits);
  const int64_t s0 = sl * each, s1 = s0 + each < steps ? s0 + each : steps;
  const int64_t cols = head_cols(p.vocab);
  const Operand A{p.weight, p.ldw, p.dim, p.vocab};
  const Operand B{p.e, cols, n, cols};
  f32x4_t acc[8][NB];
  // (a cut that leaves the last slice empty is left out by the rows above: each >= 1)
  tile_loop<TN, kWavesB, true, false, POW>(acc, lds, A, td * kTileA, B, tt * TN,
                                           s0 < steps ? s0 : steps - 1, s1,
                                           Shift{p.shift, p.rows});

  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv & 1, wn = wv >> 1;
#pragma unroll
  for (int t = 0; t < NB; ++t) {
    const int in = 16 * (NB * wn + t) + j, row = (int)(tt * TN) + in;
    if (row >= n) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t col = td * kTileA + 128 * wm + 32 * i + 8 * g;
      float o[8];
      eight<NB>(acc, i, t, g, o);
      if (splits > 1) {
        if (s0 >= steps) {
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = 0.f;
        }
        float4* to = reinterpret_cast<float4*>(part + ((sl * na + td) * nb + tt) * (TN * kTileA) +
                                               in * kTileA + 128 * wm + 32 * i + 8 * g);
        to[0] = make_float4(o[0], o[1], o[2], o[3]);
        to[1] = make_float4(o[4], o[5], o[6], o[7]);
      } else if (col < p.dim) {
        finish_row(p, POW, p.row0 + row, col, o);
        *reinterpret_cast<uint4*>(dh + p.r.src[p.row0 + row] * ldd + col) = pack8(o);
      }
    }
  }
}

// Adds the slices and rounds once: a wave 64 x 8 values of the rows, every fourth
// slice a wave and then the four in order.
__global__ __launch_bounds__(kThreads) void k_head_dh_sum(HeadPanel p, int TN, int pow,
                                                          const float* part, uint16_t* dh,
                                                          int64_t ldd) {
  __shared__ float4 buf[3][2][64];
  const int n = panel_rows(p), splits = panel_splits(p, n);
  const int64_t na = ceil_div(p.dim, kTileA), nb = ceil_div(n, TN);
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, per = p.dim / 8;
  const int64_t k = (int64_t)blockIdx.x * 64 + lane;
  if (splits == 1 || (int64_t)blockIdx.x * 64 >= (int64_t)n * per) return;
  const int64_t row = k / per;
  const int col = (int)(k - row * per) * 8;
  const bool in = row < n;
  float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto add = [&](const float4& a, const float4& b) {
    o[0] += a.x; o[1] += a.y; o[2] += a.z; o[3] += a.w;
    o[4] += b.x; o[5] += b.y; o[6] += b.z; o[7] += b.w;
  };
  if (in) {
    const float* from = part + ((col / kTileA) * nb + row / TN) * (TN * kTileA) +
                        (row % TN) * kTileA + col % kTileA;
    const int64_t step = na * nb * (TN * kTileA);
#pragma unroll 8
    for (int s = wv; s < splits; s += 4)
      add(*reinterpret_cast<const float4*>(from + s * step),
          *reinterpret_cast<const float4*>(from + s * step + 4));
  }
  if (wv > 0) {
    buf[wv - 1][0][lane] = make_float4(o[0], o[1], o[2], o[3]);
    buf[wv - 1][1][lane] = make_float4(o[4], o[5], o[6], o[7]);
  }
  __syncthreads();
  if (wv > 0 || !in) return;
#pragma unroll
  for (int w = 0; w < 3; ++w) add(buf[w][0][lane], buf[w][1][lane]);
  finish_row(p, pow, p.row0 + row, col, o);
  *reinterpret_cast<uint4*>(dh + p.r.src[p.row0 + row] * ldd + col) = pack8(o);
}

// ------------------------------------------------------------------------ dW
// A vocabulary row's gradient is often its targets' and little else, so its dz's
// rounding to bf16 would be as large as the output's own (2.6e-3 of dW's norm against
// 1.7e-3), and targets of one weight and small p all round to the same side (of 1020
// rows' mean by 2^-8).  What it leaves out is added in float32.  A workgroup per packed
// row (at work where that row is its target's last) or, if those are fewer, per
// vocabulary entry, and some columns: it looks through the panel's labels for the
// target's rows, and adds what it has found where its list has no room for as many
// labels as it has threads.  A wave adds 512 columns of every WAYS-th row of the list:
// of all, where labels have few rows (200 rows of one of 32000 cost nothing that shows;
// 2048 of one, a chain of loads, 200 us at D = 4096); of every sixteenth, where the panel
// has kRestMany rows a vocabulary entry or more (8192 rows' whole call at D = 4096: 2
// entries 312 us, 686 with all; 30 entries 232 and 268; 100 entries 246 and 236).
__device__ __forceinline__ int64_t rest_slot(const HeadPanel& p, int64_t v, int64_t q) {
  return p.rows < p.vocab ? q - p.row0 : v;
}
constexpr int kRestMany = 128;
template <int WAYS, int THREADS>
__global__ __launch_bounds__(THREADS) void k_head_rest(HeadPanel p, float* rest) {
  constexpr int kWaves = THREADS / 64, kList = 2 * THREADS, kColumns = kWaves / WAYS * 512;
  __shared__ int found[kList];
  __shared__ float off[kList];
  __shared__ int wave_count[kWaves];
  __shared__ __attribute__((aligned(16))) float sums[WAYS > 1 ? kWaves : 1][WAYS > 1 ? 512 : 1];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int n = panel_rows(p);
  int self, y;                           // the target and the last row with it
  if (p.rows < p.vocab) {
    self = blockIdx.x;
    if (self >= n) return;
    y = p.r.y[p.row0 + self];
    if (y < 0 || p.r.last[y] != p.row0 + self) return;
  } else {
    y = blockIdx.x;
    self = (int)(p.r.last[y] - p.row0);
    if (self < 0) return;                // (of an earlier panel, or none)
  }
  const int way = wv % WAYS, col = (int)blockIdx.y * kColumns + wv / WAYS * 512 + lane * 8;
  float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  int have = 0;
  for (int t0 = 0; t0 <= self; t0 += THREADS) {
    const int t = t0 + tid;
    const bool hit = t <= self && p.r.y[p.row0 + t] == y;
    const uint64_t m = __builtin_amdgcn_ballot_w64(hit);
    if (lane == 0) wave_count[wv] = __popcll(m);
    __syncthreads();
    int at = have + __popcll(m & ((1ull << lane) - 1));
    for (int w = 0; w < kWaves; ++w) {
      if (w < wv) at += wave_count[w];
      have += wave_count[w];
    }
    if (hit) {
      const float c = p.r.scale[p.row0 + t].c;
      found[at] = t;
      off[at] = c - bf16_to_f32((uint16_t)pack_bf16x2(c, 0.f));
    }
    __syncthreads();
    if (have + THREADS <= kList && t0 + THREADS <= self) continue;
    if (col < p.dim) {
#pragma unroll 8
      for (int k = way; k < have; k += WAYS) {
        const uint4 h =
            *reinterpret_cast<const uint4*>(p.r.h + (p.row0 + found[k]) * p.dim + col);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          o[e] += off[k] * bf16_to_f32((uint16_t)((&h.x)[e >> 1] >> (16 * (e & 1))));
      }
    }
    have = 0;
    __syncthreads();
  }
  if constexpr (WAYS > 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[wv][lane + 64 * e] = o[e];
    __syncthreads();
    if (way > 0) return;
#pragma unroll
    for (int w = 1; w < WAYS; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] += sums[wv + w][lane + 64 * e];
  }
  if (col >= p.dim) return;
  float4* to =
      reinterpret_cast<float4*>(rest + rest_slot(p, y, p.row0 + self) * p.dim + col);
  to[0] = make_float4(o[0], o[1], o[2], o[3]);
  to[1] = make_float4(o[4], o[5], o[6], o[7]);
}

// A = h (transposed by the reads), B = dz (likewise); inner index the rows.  Bound by
// the matrix cores, and by 1 GB of writes at V = 128256, D = 4096: 2048 rows 1.91 to 2.0 ms,
// 1080 to 1130 TF (torch's product of that layout reaches 1059).
__global__ __attribute__((amdgpu_flat_work_group_size(128 * kWavesB, 128 * kWavesB),
                          amdgpu_waves_per_eu(kWavesB / 2, kWavesB / 2)))
void k_head_dw(HeadPanel p, const float* rest, int splits, float* part, float* sum, int first,
               int last, uint16_t* dw, int64_t ldo) {
  constexpr int TN = 256, NB = Shape<TN, kWavesB>::kTilesB;
  __shared__ __attribute__((aligned(1024))) char lds[Shape<TN, kWavesB>::kLds];
  const int n = panel_rows(p);
  const int64_t na = ceil_div(p.dim, kTileA), nb = ceil_div(p.vocab, TN);
  int64_t td, tv;
  int sl;
  if (!tile_of(blockIdx.x, na, nb, td, tv, splits, &sl)) return;
  const int64_t cols = head_cols(p.vocab), steps = ceil_div(n, kStep);
  const int64_t each = ceil_div(steps, splits), s0 = sl * each;
  const int64_t s1 = s0 + each < steps ? s0 + each : steps;
  if (splits > 1 && s0 >= s1) return;      // (k_head_dw_sum leaves it out)
  const Operand A{p.r.h + p.row0 * p.dim, p.dim, p.dim, steps * kStep};
  const Operand B{p.e, cols, cols, steps * kStep};
  f32x4_t acc[8][NB];
  if (steps > 0) {
    tile_loop<TN, kWavesB, true, true>(acc, lds, A, td * kTileA, B, tv * TN, s0, s1);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int t = 0; t < NB; ++t) {
        acc[i][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        asm volatile("" : "+a"(acc[i][t]));
      }
    mfma_settle();
  }
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv & 1, wn = wv >> 1;
#pragma unroll
  for (int t = 0; t < NB; ++t) {
    const int64_t v = tv * TN + 16 * (NB * wn + t) + j;
    if (v >= p.vocab) continue;
    if (splits > 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float o[8];
        eight<NB>(acc, i, t, g, o);
        float4* to = reinterpret_cast<float4*>(part + ((sl * na + td) * nb + tv) * (TN * kTileA) +
                                               (v - tv * TN) * kTileA + 128 * wm + 32 * i + 8 * g);
        to[0] = make_float4(o[0], o[1], o[2], o[3]);
        to[1] = make_float4(o[4], o[5], o[6], o[7]);
      }
      continue;
    }
    const int row = p.r.last[v];         // (of an earlier panel: none here)
    const float* add = row < p.row0 ? nullptr : rest + rest_slot(p, v, row) * p.dim;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t col = td * kTileA + 128 * wm + 32 * i + 8 * g;
      if (col >= p.dim) continue;
      float o[8];
      eight<NB>(acc, i, t, g, o);
      if (add) {
        const float4 a = *reinterpret_cast<const float4*>(add + col);
        const float4 b = *reinterpret_cast<const float4*>(add + col + 4);
        o[0] += a.x; o[1] += a.y; o[2] += a.z; o[3] += a.w;
        o[4] += b.x; o[5] += b.y; o[6] += b.z; o[7] += b.w;
      }
      if (sum) {
        float4* at = reinterpret_cast<float4*>(sum + v * p.dim + col);
        if (!first) {
          const float4 a = at[0], b = at[1];
          o[0] += a.x; o[1] += a.y; o[2] += a.z; o[3] += a.w;
          o[4] += b.x; o[5] += b.y; o[6] += b.z; o[7] += b.w;
        }
        if (!last) {
          at[0] = make_float4(o[0], o[1], o[2], o[3]);
          at[1] = make_float4(o[4], o[5], o[6], o[7]);
        }
      }
      if (last) *reinterpret_cast<uint4*>(dw + v * ldo + col) = pack8(o);
    }
  }
}

// Few tiles of dW: its rows were cut over the CUs; a thread 8 values.
__global__ __launch_bounds__(kThreads) void k_head_dw_sum(HeadPanel p, const float* rest, int splits,
                                                          const float* part, uint16_t* dw,
                                                          int64_t ldo) {
  const int n = panel_rows(p);
  const int64_t na = ceil_div(p.dim, kTileA), nb = ceil_div(p.vocab, kTileA);
  const int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int per = p.dim / 8;
  const int64_t v = k / per;
  const int col = (int)(k - v * per) * 8;
  if (v >= p.vocab) return;
  const int64_t steps = ceil_div(n, kStep), each = ceil_div(steps, splits);
  const int used = each > 0 ? (int)ceil_div(steps, each) : 0;
  float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto add = [&](const float* x) {
    const float4 a = *reinterpret_cast<const float4*>(x);
    const float4 b = *reinterpret_cast<const float4*>(x + 4);
    o[0] += a.x; o[1] += a.y; o[2] += a.z; o[3] += a.w;
    o[4] += b.x; o[5] += b.y; o[6] += b.z; o[7] += b.w;
  };
  const float* from = part + ((col / kTileA) * nb + v / kTileA) * (kTileA * kTileA) +
                      (v % kTileA) * kTileA + col % kTileA;
#pragma unroll 4
  for (int s = 0; s < used; ++s) add(from + s * (na * nb * (kTileA * kTileA)));
  const int row = p.r.last[v];
  if (row >= p.row0) add(rest + rest_slot(p, v, row) * p.dim + col);
  *reinterpret_cast<uint4*>(dw + v * ldo + col) = pack8(o);
}

// Slices of an inner index of `steps` where `tiles` tiles leave CUs without one, none
// of them empty, each of four steps or more: the parts cost about as much.
int few_tiles_splits(int64_t tiles, int64_t steps) {
  int64_t s = 256 / (tiles > 0 ? tiles : 1);
  s = s < steps / 4 ? s : steps / 4;
  s = s < 32 ? s : 32;
  if (s < 2) return 1;
  return (int)ceil_div(steps, ceil_div(steps, s));
}
int logits_splits(int64_t rows, int dim, int64_t vocab, int tile) {
  return few_tiles_splits(ceil_div(vocab, kTileA) * ceil_div(rows, tile), dim / kStep);
}
int dw_splits(int64_t rows, int dim, int64_t vocab) {
  return few_tiles_splits(ceil_div(dim, kTileA) * ceil_div(vocab, kTileA), ceil_div(rows, kStep));
}

unsigned grid8(int64_t tiles) { return (unsigned)(ceil_div(tiles, 8) * 8); }

template <int TN, int MODE>
hipError_t start_logits(const HeadPanel& p, dim3 grid, int splits, float* part, hipStream_t s) {
  constexpr int WB = logits_waves(TN, MODE);
  return launch_kernel(k_head_logits<TN, MODE, WB>, grid, dim3(128 * WB), s, p, splits, part);
}

template <int TN>
hipError_t launch_logits(const HeadPanel& p, int mode, int splits, float* part, hipStream_t s) {
  const dim3 grid(grid8(ceil_div(p.vocab, kTileA) * ceil_div(p.rows, TN) * splits));
  switch (splits > 1 ? HEAD_RAW : mode) {
    case HEAD_STATS: return start_logits<TN, HEAD_STATS>(p, grid, 1, part, s);
    case HEAD_EXP: return start_logits<TN, HEAD_EXP>(p, grid, 1, part, s);
    case HEAD_DZ: return start_logits<TN, HEAD_DZ>(p, grid, 1, part, s);
    case HEAD_POW: return start_logits<TN, HEAD_POW>(p, grid, 1, part, s);
    default: break;
  }
  const hipError_t e = start_logits<TN, HEAD_RAW>(p, grid, splits, part, s);
  if (e != hipSuccess) return e;
  const dim3 g2((unsigned)ceil_div(p.rows, 4), (unsigned)(2 * ceil_div(p.vocab, kTileA)));
  const dim3 b2(kThreads);
  switch (mode) {
    case HEAD_STATS: return launch_kernel(k_head_slices<HEAD_STATS>, g2, b2, s, p, TN, splits, part);
    case HEAD_EXP: return launch_kernel(k_head_slices<HEAD_EXP>, g2, b2, s, p, TN, splits, part);
    case HEAD_DZ: return launch_kernel(k_head_slices<HEAD_DZ>, g2, b2, s, p, TN, splits, part);
    default: return launch_kernel(k_head_slices<HEAD_POW>, g2, b2, s, p, TN, splits, part);
  }
}

// Workgroups of dh, and tiles of its partial sums, that any number of rows up to
// the panel's can ask for.
struct DhSize {
  int64_t grid, slots;
};
DhSize dh_size(int64_t rows, int dim, int64_t vocab, int tile) {
  const int64_t na = ceil_div(dim, kTileA), steps = ceil_div(vocab, kStep);
  const int64_t all = ceil_div(rows, tile);
  DhSize d{ceil_div(na * all, 8) * 8, 0};   // uncut
  for (int64_t nb = 1; nb <= all && na * nb <= kMaxSlots; ++nb) {
    const int64_t sp = dh_splits(na * nb, steps);
    if (ceil_div(na * nb * sp, 8) * 8 > d.grid) d.grid = ceil_div(na * nb * sp, 8) * 8;
    if (sp > 1 && na * nb * sp > d.slots) d.slots = na * nb * sp;
  }
  return d;
}

}  // namespace

int head_dh_splits(int64_t rows, int dim, int64_t vocab, int tile) {
  return dh_splits(ceil_div(dim, kTileA) * ceil_div(rows, tile), ceil_div(vocab, kStep));
}

int head_tile(int64_t rows, int64_t vocab) {
  // The least time of the logits' rounds: a round of 256 workgroups takes about 45, 65
  // and 118 us at 4096 inner indices with tiles of 64, 128 and 256 rows.  (331 rows
  // of a vocabulary of 128256: 555, 393 and 474 us; 700 rows: 1162, 726 and 663; 96
  // rows of 32000 at 1024: 25, 26 and 34.)  How many rows have a target only the GPU
  // knows: the mean over all of them and five in eight.
  const int unit[3] = {45, 65, 118};
  const int64_t all = rows > 0 ? rows : 1, some = ceil_div(5 * all, 8);
  int best = 64;
  int64_t least = -1;
  for (int i = 0; i < 3; ++i) {
    const int tile = 64 << i;
    const int64_t nv = ceil_div(vocab, kTileA);
    const int64_t cost = unit[i] * (ceil_div(ceil_div(all, tile) * nv, 256) +
                                    ceil_div(ceil_div(some, tile) * nv, 256));
    if (least < 0 || cost < least) {
      least = cost;
      best = tile;
    }
  }
  return best;
}

hipError_t launch_head_pack(const HeadPackArgs& a, hipStream_t s) {
  // (a workgroup also without rows: it writes how many there are)
  const int64_t per = a.rows > 512 ? ceil_div(a.rows, 512) : 1;
  const int64_t groups = a.rows > 0 ? ceil_div(a.rows, per) : 1;
  return launch_kernel(k_head_pack, dim3((unsigned)groups), dim3(kThreads), s, a, per);
}

size_t head_logits_floats(int64_t rows, int dim, int64_t vocab, int tile) {
  const int sp = logits_splits(rows, dim, vocab, tile);
  return sp > 1 ? (size_t)sp * ceil_div(vocab, kTileA) * ceil_div(rows, tile) * tile * kTileA : 0;
}

hipError_t launch_head_logits(const HeadPanel& p, int tile, int mode, float* part, hipStream_t s) {
  const int splits = logits_splits(p.rows, p.dim, p.vocab, tile);
  return tile == 64    ? launch_logits<64>(p, mode, splits, part, s)
         : tile == 128 ? launch_logits<128>(p, mode, splits, part, s)
                       : launch_logits<256>(p, mode, splits, part, s);
}

hipError_t launch_head_join(const HeadPanel& p, int kind, int shift, double* lp, float* logp,
                            HeadStat* stat, hipStream_t s) {
  return launch_kernel(k_head_join, dim3((unsigned)ceil_div(p.rows, kJoinRows)),
                       dim3(64 * kJoinWaves), s,
                       p, kind, shift, lp, logp, stat);
}

hipError_t launch_head_loss(const int32_t* n, const double* lp, int mean, float* loss,
                            hipStream_t s) {
  return launch_kernel(k_head_loss, dim3(1), dim3(1024), s, n, lp, mean, loss);
}

hipError_t launch_head_dz(const HeadPanel& p, hipStream_t s) {
  const dim3 grid((unsigned)(p.rows / kDzRows),
                  (unsigned)ceil_div(head_cols(p.vocab), kThreads * 8));
  return launch_kernel(k_head_dz, grid, dim3(kThreads), s, p);
}

size_t head_dh_floats(int64_t rows, int dim, int64_t vocab, int tile) {
  return (size_t)dh_size(rows, dim, vocab, tile).slots * tile * kTileA;
}

template <bool POW>
hipError_t launch_dh(const HeadPanel& p, int tile, dim3 grid, float* part, uint16_t* dh,
                     int64_t ldd, hipStream_t s) {
  const dim3 block(128 * kWavesB);
  return tile == 64    ? launch_kernel(k_head_dh<64, POW>, grid, block, s, p, part, dh, ldd)
         : tile == 128 ? launch_kernel(k_head_dh<128, POW>, grid, block, s, p, part, dh, ldd)
                       : launch_kernel(k_head_dh<256, POW>, grid, block, s, p, part, dh, ldd);
}
hipError_t launch_head_dh(const HeadPanel& p, int tile, int pow, float* part, uint16_t* dh,
                          int64_t ldd, hipStream_t s) {
  const DhSize d = dh_size(p.rows, p.dim, p.vocab, tile);
  const dim3 grid((unsigned)d.grid);
  const hipError_t e = pow ? launch_dh<true>(p, tile, grid, part, dh, ldd, s)
                           : launch_dh<false>(p, tile, grid, part, dh, ldd, s);
  if (e != hipSuccess || d.slots == 0) return e;
  // (rows of more tiles than kMaxSlots are not cut)
  const int64_t most = kMaxSlots / ceil_div(p.dim, kTileA) * tile;
  const int64_t rows = p.rows < most ? p.rows : most;
  return launch_kernel(k_head_dh_sum, dim3((unsigned)ceil_div(rows * p.dim / 8, 64)),
                       dim3(kThreads), s, p, tile, pow, part, dh, ldd);
}

hipError_t launch_head_rest(const HeadPanel& p, float* rest, hipStream_t s) {
  const unsigned slots = (unsigned)head_slots(p.rows, p.vocab);
  return p.rows >= kRestMany * p.vocab
             ? launch_kernel(k_head_rest<16, 1024>, dim3(slots, (unsigned)ceil_div(p.dim, 512)),
                             dim3(1024), s, p, rest)
             : launch_kernel(k_head_rest<1, kThreads>, dim3(slots, (unsigned)ceil_div(p.dim, 2048)),
                             dim3(kThreads), s, p, rest);
}

size_t head_dw_floats(int64_t rows, int dim, int64_t vocab) {
  const int sp = dw_splits(rows, dim, vocab);
  return sp > 1 ? (size_t)sp * ceil_div(dim, kTileA) * ceil_div(vocab, kTileA) * kTileA * kTileA : 0;
}

hipError_t launch_head_dw(const HeadPanel& p, const float* rest, float* part, float* acc, int first,
                          int last, uint16_t* dw, int64_t ldo, hipStream_t s) {
  const int splits = acc ? 1 : dw_splits(p.rows, p.dim, p.vocab);
  const dim3 grid(grid8(ceil_div(p.dim, kTileA) * ceil_div(p.vocab, kTileA) * splits));
  const hipError_t e = launch_kernel(k_head_dw, grid, dim3(128 * kWavesB), s, p, rest, splits,
                                     part, acc, first, last, dw, ldo);
  if (e != hipSuccess || splits == 1) return e;
  return launch_kernel(k_head_dw_sum, dim3((unsigned)ceil_div(p.vocab * p.dim / 8, kThreads)),
                       dim3(kThreads), s, p, rest, splits, part, dw, ldo);
}

}  // namespace qnf4
