// Arguments and launchers of the Muon kernels (muon_momentum.cu,
// muon_ns.cu) behind the mua_muon_* entry points (muon_api.cu).
//
// One step for a matrix with gradient g and momentum m (held quantized):
//   m' = beta m + g,  U = g + beta m' (Nesterov) or m'
//   X_0 = U / (|U|_F + eps),  X_{k+1} = (a I + b A + c A^2) X_k,  A = X_k X_k^T
//   p <- p (1 - lr wd) - lr scale X_steps
// with A on the short side (X_k^T X_k for a tall matrix, X_{k+1} = X_k P).
//
// Number formats of the iteration. X, A and P = a I + b A + c A^2 are stored
// in fp16 (11 significant bits) with a power of two that the host derives
// from a bound on their spectral norms, so that no entry overflows and an
// entry is subnormal only when it is 2^-28 of that bound; every product and
// norm is summed in fp32 or fp64. Against fp64, simulated for a Gaussian matrix
// of 768 x 768: 1.2e-3 relative in the Frobenius norm (bf16 operands: 1.0e-2;
// the final rounding to bf16 alone: 1.7e-3). Matrices that stay on one SM hold A
// and P as two fp16 values each: 0.5e-3 for long ones, 0.8e-3 to 1e-3 for square
// ones. Where the singular values lie close together, as of a long Gaussian matrix
// of few rows, the diagonals of A and P round alike and the errors add up: 2.2e-3
// for 26 x 8319.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mua {

constexpr int kMuonBlock = 128;          // values per quantization scale
constexpr int kMuonMaxSteps = 16;
constexpr int kMuonHdrStatus = 4;        // header word, as in the MicroAdam state
constexpr uint32_t kMuonNonFinite = 1u;
constexpr uint32_t kMuonTimeout = 2u;

enum MuonType : int { kF32 = 0, kBf16 = 1 };

// A stack of `count` row-major matrices: element (i, r, c) at
// p + (i matrix_stride + r row_stride + c) * size.
struct MuonView {
  void* p;
  int type;
  int64_t matrix_stride, row_stride;
};

struct MuonShape {
  int32_t rows, cols, count;  // count: matrices of this launch
  int32_t ld;                 // row stride of the fp16 matrices X
  int32_t parts;              // partial sums per matrix
};

struct MuonQuant {
  int32_t bits;               // 8 or 4
  int64_t bpm;                // blocks of one matrix
  float* scales;              // of the launch's first matrix
  uint8_t* codes;
  uint32_t* status;
};

struct MuonRandom {
  uint32_t t_lo, t_hi;
  uint32_t keys[10][2];       // Philox round keys
  int64_t base;               // global index of the launch's first value
};

// Sum of squares of x (or of the direction U) per matrix and part.
cudaError_t muon_launch_norm(const MuonShape& s, const MuonView& x, double* partials,
                             cudaStream_t st);
cudaError_t muon_launch_direction_norm(const MuonShape& s, const MuonQuant& q, const void* g,
                                       int g_type, float beta, int nesterov, double* partials,
                                       cudaStream_t st);
// X_0 in fp16: x 2^(e0 - t) with 2^(t-1) <= |x|_F + eps < 2^t, an exact scaling;
// factor[i] = 2^t / (|x|_F + eps) is applied in fp32 by the first products.
// Both also zero the matrices' counters.
cudaError_t muon_launch_load(const MuonShape& s, const MuonView& x, const double* partials,
                             float eps, int e0, void* X, float* factor, uint32_t* counters,
                             cudaStream_t st);
// The momentum update; direction U to `out` (fp32 or bf16, contiguous), or,
// with X != NULL, straight to X_0 as in muon_launch_load.
cudaError_t muon_launch_momentum(const MuonShape& s, const MuonQuant& q, const void* g, int g_type,
                                 float beta, int nesterov, const MuonRandom& rnd, void* out,
                                 int out_type, const double* partials, float eps, int e0, void* X,
                                 float* factor, uint32_t* counters, cudaStream_t st);
cudaError_t muon_launch_read(const MuonShape& s, const MuonQuant& q, void* out, int out_type,
                             cudaStream_t st);
cudaError_t muon_launch_write(const MuonShape& s, const MuonQuant& q, const void* values, int type,
                              cudaStream_t st);

// ---------------------------------------------------------------- products
struct MuonNs {
  int32_t rows, cols, batch, steps;
  // fp16 matrices: X [batch][rows][ld] of even and odd steps (X_0 in x[0]); A and
  // P [batch][s][lds], s the short side.
  void* x[2];
  void *a, *p;
  int32_t ld, lds;
  // Items that share a tile of A's contraction and that add the shares up (a
  // power of two up to 16); fp32 [batch][tile][split][256 or 128 squared].
  int32_t split, reduce;
  float* partials;
  // Power-of-two scales and coefficients of each step's products.
  float gram_alpha[kMuonMaxSteps];
  float poly_alpha[kMuonMaxSteps], poly_mid[kMuonMaxSteps], poly_diag[kMuonMaxSteps];
  float update_alpha[kMuonMaxSteps];  // of the last: lr scale, or the result's
  const float* factor;         // per matrix, applied in step 0
  // The last product: result (bf16) or parameters p <- p decay - alpha x.
  void* out;
  int64_t ldo, batch_stride;   // in elements
  int32_t params, out_type, out_vec;
  float decay;
  uint32_t* counters;          // per matrix: finished parts of tiles, 0 at the launch
  uint32_t* status;
  uint64_t wait_ns;            // longest wait inside the kernel before it gives up
};

// On output tiles of bn = 256 (CTA pairs) or 128.
cudaError_t muon_launch_ns(const MuonNs& g, int bn, cudaStream_t st);

// Matrices that fit a CTA's shared memory: the whole operator in one launch, a
// CTA each. Shared memory it takes, 0 where a matrix does not fit.
uint32_t muon_small_smem(int32_t rows, int32_t cols);
cudaError_t muon_launch_small(const MuonShape& s, const MuonNs& g, const MuonView& x, float eps,
                              int e0, cudaStream_t st);
cudaError_t muon_launch_small_step(const MuonShape& s, const MuonNs& g, const MuonQuant& q,
                                   const void* grads, int g_type, float beta, int nesterov,
                                   const MuonRandom& rnd, float eps, int e0, cudaStream_t st);

}  // namespace mua
