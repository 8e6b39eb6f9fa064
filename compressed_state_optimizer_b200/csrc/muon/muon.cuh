// Arguments and launchers of the Muon kernels (muon_momentum.cu,
// muon_gemm.cu) behind the mua_muon_* entry points (muon_api.cu).
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
// norm is summed in fp32 or fp64. Against fp64, for a Gaussian matrix of
// 768 x 768: 1.2e-3 relative in the Frobenius norm (bf16 operands: 1.0e-2;
// the final rounding to bf16 alone: 1.7e-3).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mua {

constexpr int kMuonBlock = 128;          // values per quantization scale
constexpr int kMuonMaxSteps = 16;
constexpr int kMuonMaxParts = 256;       // partial sums of one matrix's norm
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
  int32_t ld;                 // row stride of the fp16 matrices X (cols up to a multiple of 8)
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
cudaError_t muon_launch_load(const MuonShape& s, const MuonView& x, const double* partials,
                             float eps, int e0, void* X, float* factor, cudaStream_t st);
// The momentum update; direction U to `out` (fp32 or bf16, contiguous), or,
// with X != NULL, straight to X_0 as in muon_launch_load.
cudaError_t muon_launch_momentum(const MuonShape& s, const MuonQuant& q, const void* g, int g_type,
                                 float beta, int nesterov, const MuonRandom& rnd, void* out,
                                 int out_type, const double* partials, float eps, int e0, void* X,
                                 float* factor, cudaStream_t st);
cudaError_t muon_launch_read(const MuonShape& s, const MuonQuant& q, void* out, int out_type,
                             cudaStream_t st);
cudaError_t muon_launch_write(const MuonShape& s, const MuonQuant& q, const void* values, int type,
                              cudaStream_t st);

// ---------------------------------------------------------------- products
enum MuonEpilogue : int {
  kGram = 0,    // A = alpha f^2 X X^T
  kPoly = 1,    // P = diag I + mid A + alpha A A
  kUpdate = 2,  // X' = alpha f P X, fp16
  kOut = 3,     // alpha f P X to a bf16 stack
  kParams = 4,  // p <- p decay - alpha f (P X)
};

struct MuonGemm {
  int32_t M, N, K, batch;      // D [M x N] per matrix
  int32_t tiles_m, tiles_n, tiles;  // tiles: of one matrix
  float alpha, mid, diag, decay;
  const float* factor;         // per matrix, NULL: 1
  const void* addend;          // A (kPoly)
  void* out;                   // fp16 [batch][M][ldo], or the caller's stack
  int64_t ldo, batch_stride;   // in elements
  int32_t out_type;            // of kOut / kParams
  int32_t out_vec;             // 16-byte accesses allowed on the caller's stack
  uint32_t* status;
  uint64_t wait_ns;            // longest wait inside the kernel before it gives up
};

struct MuonOperand {
  void* p;                     // fp16 [batch][rows][ld]
  int32_t rows, cols, ld;
};

// D = op(A) op(B): an operand whose contraction index is contiguous ("K-major")
// or whose M / N index is (`mn`).
cudaError_t muon_launch_gemm(const MuonOperand& a, bool a_mn, const MuonOperand& b, bool b_mn,
                             int epilogue, MuonGemm g, cudaStream_t st);

int muon_sm_count(cudaError_t* e);

}  // namespace mua
