// Launcher interface of the orthogonalised update (Newton-Schulz products).
#pragma once

#include "nf4_common.h"

namespace qnf4 {

// One matrix: `in` is the gradient (of a step) or the update itself; m the momentum
// (null: none); `out` the parameter of a step, with its bf16 copy pb (nullable), or
// what receives the orthogonalised matrix.  Row strides in elements.
struct MuonTensor {
  const void* in;
  float* m;
  void* out;
  uint16_t* pb;
  int32_t rows, cols;
  int32_t ldi, ldm, ldo, ldb;
  float scale;        // of a step: lr times the shape's factor
  int32_t bf16;       // type of `in` (and of `out` without a step)
  int32_t wg, slice;  // its first slice in the call, long indices of each
  int32_t chunk;      // its first chunk in the call
  uint32_t part, q;   // its partial products and polynomial, in tiles of 256 doubles
  int32_t reserved;
};
constexpr int kMuonBatch = 45;   // per launch: 3.9 KB of kernel arguments
struct MuonBatch {
  int count, first;              // index of t[0] in the call
  MuonTensor t[kMuonBatch];
};
struct MuonHyper {
  float mu, one_minus_mu, decay;
  int nesterov, step, steps;     // step: update parameters; else write the matrix
  double a, b, c, eps;
};
struct MuonScratch {
  MuonTensor* t;                 // [tensors]
  int32_t* owner;                // [chunks] tensor of each
  int32_t* owner_wg;             // [slices] likewise
  double* part;
  double* q;
};

// Padded short side (16, 32, 64 or 128), long indices of a chunk, and 16 x 16 tiles of
// the products' upper triangle.
inline __host__ __device__ int muon_pad(int s) {
  return s <= 16 ? 16 : s <= 32 ? 32 : s <= 64 ? 64 : 128;
}
inline __host__ __device__ int muon_chunk(int sp) { return 4096 / sp; }
inline __host__ __device__ int muon_tiles(int sp) { return (sp / 16) * (sp / 16 + 1) / 2; }
// Long indices of a workgroup, for a call of `total` elements.
int muon_slice(int sp, int64_t total);

// Chunks of a matrix that one workgroup can take whole, where its padded short side is
// 32 or less, and the update of a batch of nothing else (those of that short side).
constexpr int kMuonSmall = 4;
hipError_t launch_muon_small(const MuonBatch& b, int sp, const MuonHyper& h, hipStream_t st);
// Tensors of a batch to the scratch's table.
hipError_t launch_muon_table(const MuonBatch& b, const MuonScratch& s, hipStream_t st);
// m, and the slices' products of the tensors whose padded short side is sp: those of
// the table (b null), or of a batch that is the whole call, which goes to the table
hipError_t launch_muon_gram(const MuonBatch* b, int sp, int wgs, const MuonHyper& h,
                            const MuonScratch& s, hipStream_t st);
// polynomials, then the update, of the call's tensors of that padded short side
hipError_t launch_muon_poly(int count, int sp, const MuonHyper& h, const MuonScratch& s,
                            hipStream_t st);
hipError_t launch_muon_apply(int sp, int chunks, const MuonHyper& h, const MuonScratch& s,
                             hipStream_t st);

}  // namespace qnf4
