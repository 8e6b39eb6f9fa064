// Host side of the mua_muon_* entry points declared in include/mua.h.
//
// A handle holds geometry and the polynomial's plan only. A step runs the
// stack in groups of matrices (one X of a group takes at most kGroupBytes, half of
// the L2; both X, A and P together may be more) and enqueues, per group: the norm of the direction, the momentum update
// with X_0, and the Newton-Schulz steps in one launch whose last product
// updates the parameters. No device memory is allocated and nothing is synchronized.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <new>

#include "../../../include/mua.h"
#include "muon.cuh"

static_assert(MUA_F32 == mua::kF32 && MUA_BF16 == mua::kBf16, "type codes");
static_assert(MUA_STATUS_NONFINITE == mua::kMuonNonFinite &&
                  MUA_STATUS_TIMEOUT == mua::kMuonTimeout,
              "status bits");

struct Tiling {               // of the products: see tiling()
  int32_t bn, split, reduce;
  double us;
};

struct mua_muon_ctx {
  int32_t rows, cols, count, bits, steps;
  int32_t s;                 // short side: A and P are s x s
  bool tall;                 // rows > cols
  bool small;                // one CTA holds a matrix on chip
  int32_t ld, lds;           // fp16 row strides of X and of A, P
  int32_t group, parts;
  Tiling tiling;
  int64_t bpm;               // blocks of one matrix
  int64_t off_scales, off_codes, state_bytes;
  int64_t off_partials, off_factor, off_counters, off_x[2], off_a, off_p, off_split, workspace_bytes;
  float coef[mua::kMuonMaxSteps][3];
  int32_t ex[mua::kMuonMaxSteps + 1], ea[mua::kMuonMaxSteps], ep[mua::kMuonMaxSteps];
  int64_t wait_ns;
};

namespace {

thread_local char g_error[256] = "no CUDA error";

constexpr int64_t kDefaultWaitNs = 2000000000;
constexpr int64_t kGroupBytes = 64 << 20;  // X of one group

int fail(cudaError_t e, const char* where) {
  std::snprintf(g_error, sizeof g_error, "%s: %s", where, cudaGetErrorString(e));
  return MUA_ERR_CUDA;
}

int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool valid_type(int32_t t) { return t == MUA_F32 || t == MUA_BF16; }
int64_t type_size(int32_t t) { return t == MUA_F32 ? 4 : 2; }

// The power of two that puts a bound on every entry at 15000 .. 30000, half of
// fp16's range: entries are at most the spectral norm, and the bound itself is
// 2 % wide for the roundings of the iteration.
int exponent_for(double bound) {
  const int e = (int)std::floor(std::log2(30000.0 / bound));
  return std::max(-24, std::min(40, e));
}

// Bounds of |X_k|, |A_k| and |P_k| over singular values in [0, 1] of X_0.
bool plan(mua_muon_ctx* h) {
  double top = 1.02;
  h->ex[0] = exponent_for(top);
  for (int k = 0; k < h->steps; ++k) {
    const double a = h->coef[k][0], b = h->coef[k][1], c = h->coef[k][2];
    double next = 0.0, poly = 0.0;
    const int n = 4096;
    for (int i = 0; i <= n; ++i) {
      const double x = top * i / n, y = a + x * x * (b + x * x * c);
      poly = std::max(poly, std::fabs(y));
      next = std::max(next, std::fabs(x * y));
    }
    h->ea[k] = exponent_for(top * top);
    h->ep[k] = exponent_for(std::max(1.02 * poly, 1e-6));
    top = std::max(1.02 * next, 1e-6);
    // fp16 holds the iteration's range only while its norms stay moderate.
    if (!(top <= 1024.0) || !(poly <= 65536.0)) return false;
    h->ex[k + 1] = exponent_for(top);
  }
  return true;
}

mua::MuonShape shape(const mua_muon_ctx* h, int32_t count) {
  mua::MuonShape s;
  s.rows = h->rows;
  s.cols = h->cols;
  s.count = count;
  s.ld = h->ld;
  s.parts = h->parts;
  return s;
}

mua::MuonQuant quant(const mua_muon_ctx* h, const void* state, int32_t first) {
  uint8_t* p = static_cast<uint8_t*>(const_cast<void*>(state));
  mua::MuonQuant q;
  q.bits = h->bits;
  q.bpm = h->bpm;
  q.scales = reinterpret_cast<float*>(p + h->off_scales) + first * h->bpm;
  q.codes = p + h->off_codes + first * h->bpm * mua::kMuonBlock * h->bits / 8;
  q.status = reinterpret_cast<uint32_t*>(p) + mua::kMuonHdrStatus;
  return q;
}

mua::MuonRandom random_keys(const mua_muon_ctx* h, int32_t first, int64_t t, uint64_t seed) {
  mua::MuonRandom r;
  r.t_lo = (uint32_t)(uint64_t)t;
  r.t_hi = (uint32_t)((uint64_t)t >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
  for (int i = 0; i < 10; ++i) {
    r.keys[i][0] = k0;
    r.keys[i][1] = k1;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  r.base = first * h->bpm * mua::kMuonBlock;
  return r;
}

struct Target {  // where the last product goes
  bool params;
  void* out;
  int type;
  int64_t matrix_stride, row_stride;
  double alpha;   // lr * scale, or 1
  float decay;
};

uint32_t* counters(const mua_muon_ctx* h, uint8_t* ws) {
  return reinterpret_cast<uint32_t*>(ws + h->off_counters);
}

// The iteration of matrices first .. first + count - 1.
mua::MuonNs iteration(const mua_muon_ctx* h, int32_t first, int32_t count, const Target& to,
                      uint32_t* status) {
  mua::MuonNs g;
  std::memset(&g, 0, sizeof g);
  g.rows = h->rows;
  g.cols = h->cols;
  g.batch = count;
  g.steps = h->steps;
  for (int k = 0; k < h->steps; ++k) {
    const int ex = h->ex[k], ea = h->ea[k], ep = h->ep[k];
    const bool last = k + 1 == h->steps;
    g.gram_alpha[k] = (float)std::ldexp(1.0, ea - 2 * ex);
    g.poly_alpha[k] = (float)std::ldexp((double)h->coef[k][2], ep - 2 * ea);
    g.poly_mid[k] = (float)std::ldexp((double)h->coef[k][1], ep - ea);
    g.poly_diag[k] = (float)std::ldexp((double)h->coef[k][0], ep);
    g.update_alpha[k] = (float)(last ? std::ldexp(to.alpha, -ep - ex)
                                     : std::ldexp(1.0, h->ex[k + 1] - ep - ex));
  }
  const int64_t size = type_size(to.type);
  g.out = static_cast<uint8_t*>(to.out) + (int64_t)first * to.matrix_stride * size;
  g.ldo = to.row_stride;
  g.batch_stride = to.matrix_stride;
  g.params = to.params;
  g.out_type = to.type;
  // Four columns at a time: 16 bytes of fp32, 8 of bf16.
  g.out_vec = aligned(g.out, 4 * size) && to.row_stride % 4 == 0 &&
              (count == 1 || to.matrix_stride % 4 == 0);
  g.decay = to.decay;
  g.status = status;
  g.wait_ns = (uint64_t)std::max<int64_t>(0, h->wait_ns);
  return g;
}

// Its launch, X_0 and its factors being in the workspace.
int iterate(const mua_muon_ctx* h, uint8_t* ws, int32_t first, int32_t count, const Target& to,
            uint32_t* status, cudaStream_t st) {
  mua::MuonNs g = iteration(h, first, count, to, status);
  g.factor = reinterpret_cast<const float*>(ws + h->off_factor);
  g.counters = counters(h, ws);
  g.x[0] = ws + h->off_x[0];
  g.x[1] = ws + h->off_x[1];
  g.a = ws + h->off_a;
  g.p = ws + h->off_p;
  g.ld = h->ld;
  g.lds = h->lds;
  g.split = h->tiling.split;
  g.reduce = h->tiling.reduce;
  g.partials = reinterpret_cast<float*>(ws + h->off_split);
  const cudaError_t e = mua::muon_launch_ns(g, h->tiling.bn, st);
  return e == cudaSuccess ? MUA_OK : fail(e, "Newton-Schulz kernel launch");
}

// Time of a step's products on tiles of bn, in us: per product the waves of
// items over the SMs (whole ones for a single matrix; those of a stack overlap),
// an item's k-slices and what it adds to them, and the way from one product's
// last store to the next one's first MMA. Fitted to 36 shapes from 256 x 256 to
// 4096 x 4096 and 148 x 256 x 256, each measured on both tiles: a 64-deep slice
// takes 0.34 us on 256 x 256 tiles of CTA pairs and 0.23 us on 128 x 128, an item
// 3.0 and 1.1 us more, between products 3.3 us; the choice is within 4 % of the
// better tile on all of them. The larger one, with four times the work a slice,
// wins where its items fill the SMs anyway: 4096 x 4096 (1154 against 1494 us),
// 3000 x 3000 (545, 653), 24 x 768 x 768 (253, 316). The smaller one wins below:
// 768 x 768 (102, 142), 2048 x 2048 (218, 241), 12 x 768 x 768 (159, 181).
// Sharing A's tiles among idle SMs costs a product more: 512 x 11008 305 -> 187
// us and 1024 x 4096 199 -> 183, but 1024 x 1024 115 -> 130 us.
Tiling tiling(int32_t rows, int32_t cols, int32_t batch, int32_t bn) {
  const bool big = bn == 256;
  const double slice = big ? 0.34 : 0.23, item = big ? 3.0 : 1.1, between = 3.3;
  const int64_t units = big ? 74 : 148;  // CTA pairs or CTAs of a B200
  const int64_t s = std::min(rows, cols), l = std::max(rows, cols);
  const int64_t tm = (s + bn - 1) / bn, sym = tm * (tm + 1) / 2 * batch;
  const int64_t upd = (int64_t)((rows + bn - 1) / bn) * ((cols + bn - 1) / bn) * batch;
  const int64_t gram = (l + 63) / 64, update = (s + 63) / 64;
  auto product = [&](int64_t items, double slices) {
    const double waves = std::max(1.0, (double)items / units);
    return (batch > 1 ? waves : std::ceil(waves)) * (slices * slice + item) + between;
  };
  Tiling t = {bn, 1, 1, product(sym, gram)};
  // A share keeps 8 slices or more.
  const int64_t split = std::min<int64_t>(std::min<int64_t>(16, units / sym), gram / 8);
  if (split > 1) {
    const double us = product(sym * split, (double)gram / split) + item + between;
    if (us < t.us) {
      t.us = us;
      t.split = (int32_t)split;
      while (2 * t.reduce <= t.split) t.reduce *= 2;
    }
  }
  t.us += product(sym, update) + product(upd, update);
  return t;
}

// Row stride of an fp16 matrix in the workspace: rows start at 128-byte lines, or
// fit one, so that a copy of 64 columns never takes a part of a second line
// (1000 x 1000 at a stride of 1000: 158 us, 1024: 119; 3000 x 3000: 692, 550).
int32_t row_stride(int32_t cols) {
  if (cols > 32) return (int32_t)round_up(cols, 64);
  return cols > 16 ? 32 : cols > 8 ? 16 : 8;
}

int create(int32_t rows, int32_t cols, int32_t count, int32_t bits, int32_t steps,
           const float* coefficients, mua_muon_t* out) {
  if (!out) return MUA_ERR_ARG;
  *out = nullptr;
  if (rows < 1 || cols < 1 || count < 1 || steps < 1 || steps > MUA_MUON_MAX_STEPS)
    return MUA_ERR_ARG;
  const int64_t n = (int64_t)rows * cols;
  const int32_t s = std::min(rows, cols);
  if ((bits != 8 && bits != 4) || rows > (1 << 20) || cols > (1 << 20) || s > (1 << 15) ||
      n >= (1ll << 31))
    return MUA_ERR_UNSUPPORTED;
  const int64_t bpm = (n + mua::kMuonBlock - 1) / mua::kMuonBlock;
  if ((int64_t)count * ((bpm + 31) / 32) >= (1ll << 31)) return MUA_ERR_UNSUPPORTED;

  mua_muon_ctx* h = new (std::nothrow) mua_muon_ctx();
  if (!h) return MUA_ERR_ARG;
  h->rows = rows;
  h->cols = cols;
  h->count = count;
  h->bits = bits;
  h->steps = steps;
  for (int k = 0; k < steps; ++k)
    for (int i = 0; i < 3; ++i) {
      // The quintic whose fixed points keep every singular value of
      // [0.003, 1] within [0.67, 1.21] after five steps.
      static const float quintic[3] = {3.4445f, -4.7750f, 2.0315f};
      h->coef[k][i] = coefficients ? coefficients[3 * k + i] : quintic[i];
      if (!std::isfinite(h->coef[k][i])) {
        delete h;
        return MUA_ERR_ARG;
      }
    }
  if (!plan(h)) {
    delete h;
    return MUA_ERR_UNSUPPORTED;
  }
  h->s = s;
  h->tall = rows > cols;
  h->small = mua::muon_small_smem(rows, cols) > 0;
  h->ld = row_stride(cols);
  h->lds = row_stride(s);
  h->bpm = bpm;
  h->off_scales = 256;
  h->off_codes = h->off_scales + round_up(4ll * count * bpm, 256);
  h->state_bytes = h->off_codes + (int64_t)count * bpm * mua::kMuonBlock * bits / 8;
  h->wait_ns = kDefaultWaitNs;
  h->workspace_bytes = 256;  // the status word
  if (h->small) {  // nothing of such a matrix leaves its SM
    *out = h;
    return MUA_OK;
  }
  const int64_t x_bytes = (int64_t)rows * h->ld * 2, a_bytes = (int64_t)s * h->lds * 2;
  const int64_t items = 16 * (((int64_t)s + 127) / 128 * (((int64_t)s + 127) / 128 + 1) * 17 +
                              (((int64_t)rows + 127) / 128) * (((int64_t)cols + 127) / 128));
  const int64_t fit = std::max<int64_t>(
      1, std::min<int64_t>(std::min<int64_t>(count, kGroupBytes / x_bytes), (1 << 30) / items));
  const int64_t groups = (count + fit - 1) / fit;  // items of a launch fit 31 bits
  h->group = (int32_t)((count + groups - 1) / groups);
  const Tiling narrow = tiling(rows, cols, h->group, 128), wide = tiling(rows, cols, h->group, 256);
  h->tiling = wide.us <= narrow.us ? wide : narrow;
  // The norm's sums: four CTAs an SM of a B200 in all, 8192 values each or more.
  h->parts = (int32_t)std::max<int64_t>(
      1, std::min<int64_t>(4 * 148 / h->group, n / 8192));
  int64_t at = h->workspace_bytes;
  auto take = [&at](int64_t bytes) {
    const int64_t o = at;
    at += round_up(bytes, 256);
    return o;
  };
  h->off_partials = take((int64_t)h->group * h->parts * 8);
  h->off_factor = take((int64_t)h->group * 4);
  h->off_counters = take((int64_t)h->group * 4);
  h->off_x[0] = take(h->group * x_bytes);
  h->off_x[1] = steps > 1 ? take(h->group * x_bytes) : h->off_x[0];
  h->off_a = take(h->group * a_bytes);
  h->off_p = take(h->group * a_bytes);
  const int64_t tm = (s + h->tiling.bn - 1) / h->tiling.bn;
  h->off_split = h->tiling.split > 1
                     ? take(4ll * h->group * (tm * (tm + 1) / 2) * h->tiling.split *
                            h->tiling.bn * h->tiling.bn)
                     : at;
  h->workspace_bytes = at;
  *out = h;
  return MUA_OK;
}

bool finite_f(float x) { return std::isfinite(x); }

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// All values of a handle's stack, contiguous.
int64_t value_bytes(const mua_muon_ctx* h, int32_t type) {
  return (int64_t)h->rows * h->cols * h->count * type_size(type);
}

}  // namespace

extern "C" {

int mua_muon_create(int32_t rows, int32_t cols, int32_t count, int32_t bits, int32_t steps,
                    const float* coefficients, mua_muon_t* out) {
  return create(rows, cols, count, bits, steps, coefficients, out);
}

void mua_muon_destroy(mua_muon_t h) { delete h; }

int64_t mua_muon_state_bytes(mua_muon_t h) { return h ? h->state_bytes : MUA_ERR_ARG; }

int64_t mua_muon_workspace_bytes(mua_muon_t h) { return h ? h->workspace_bytes : MUA_ERR_ARG; }

int mua_muon_state_layout(mua_muon_t h, int64_t* out) {
  if (!h || !out) return MUA_ERR_ARG;
  out[MUA_MUON_LAYOUT_HEADER] = 0;
  out[MUA_MUON_LAYOUT_SCALES] = h->off_scales;
  out[MUA_MUON_LAYOUT_CODES] = h->off_codes;
  out[MUA_MUON_LAYOUT_BLOCKS] = h->bpm;
  out[MUA_MUON_LAYOUT_BYTES] = h->state_bytes;
  return MUA_OK;
}

int mua_muon_set_wait_limit_ns(mua_muon_t h, int64_t ns) {
  if (!h) return MUA_ERR_ARG;
  h->wait_ns = ns <= 0 ? 0 : ns;
  return MUA_OK;
}

int mua_muon_momentum(mua_muon_t h, const void* grads, int32_t grads_type, void* state,
                      void* direction, int32_t direction_type, float beta, int32_t nesterov,
                      int64_t t, uint64_t seed, void* stream) {
  if (!h || !grads || !state || !direction) return MUA_ERR_ARG;
  if (!valid_type(grads_type) || !valid_type(direction_type) || t < 1) return MUA_ERR_ARG;
  if (!(beta >= 0.0f && beta < 1.0f)) return MUA_ERR_ARG;
  if (!aligned(grads, type_size(grads_type)) || !aligned(direction, type_size(direction_type)) ||
      !aligned(state, 16))
    return MUA_ERR_ALIGN;
  const int64_t gs = value_bytes(h, grads_type), ds = value_bytes(h, direction_type);
  if (overlap(grads, gs, direction, ds) || overlap(grads, gs, state, h->state_bytes) ||
      overlap(direction, ds, state, h->state_bytes))
    return MUA_ERR_ARG;
  const cudaError_t e = mua::muon_launch_momentum(
      shape(h, h->count), quant(h, state, 0), grads, grads_type, beta, nesterov != 0,
      random_keys(h, 0, t, seed), direction, direction_type, nullptr, 0.0f, 0, nullptr, nullptr,
      nullptr,      static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MUA_OK : fail(e, "momentum kernel launch");
}

int mua_muon_read(mua_muon_t h, const void* state, void* out, int32_t type, void* stream) {
  if (!h || !state || !out || !valid_type(type)) return MUA_ERR_ARG;
  if (!aligned(state, 16) || !aligned(out, type_size(type))) return MUA_ERR_ALIGN;
  if (overlap(out, value_bytes(h, type), state, h->state_bytes)) return MUA_ERR_ARG;
  const cudaError_t e = mua::muon_launch_read(shape(h, h->count), quant(h, state, 0), out, type,
                                              static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MUA_OK : fail(e, "read kernel launch");
}

int mua_muon_write(mua_muon_t h, const void* values, int32_t type, void* state, void* stream) {
  if (!h || !state || !values || !valid_type(type)) return MUA_ERR_ARG;
  if (!aligned(state, 16) || !aligned(values, type_size(type))) return MUA_ERR_ALIGN;
  if (overlap(values, value_bytes(h, type), state, h->state_bytes)) return MUA_ERR_ARG;
  const cudaError_t e = mua::muon_launch_write(shape(h, h->count), quant(h, state, 0), values, type,
                                               static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MUA_OK : fail(e, "write kernel launch");
}

int mua_muon_orthogonalize(mua_muon_t h, const void* x, int32_t x_type, int64_t x_matrix_stride,
                           int64_t x_row_stride, void* out, int64_t out_matrix_stride,
                           int64_t out_row_stride, void* workspace, float eps, void* stream) {
  if (!h || !x || !out || !workspace || !valid_type(x_type)) return MUA_ERR_ARG;
  if (!finite_f(eps) || eps < 0.0f) return MUA_ERR_ARG;
  if (x_matrix_stride < 0 || x_row_stride < 0) return MUA_ERR_ARG;
  const int64_t row = h->cols, last = h->count - 1;
  const bool rows_ok = h->rows == 1 || out_row_stride >= row;
  const bool stacked = out_matrix_stride >= (h->rows - 1) * out_row_stride + row;
  const bool woven = out_matrix_stride >= row && out_row_stride >= last * out_matrix_stride + row;
  if (out_row_stride < 0 || out_matrix_stride < 0 || !rows_ok ||
      !(h->count == 1 || stacked || woven))
    return MUA_ERR_ARG;
  if (!aligned(x, type_size(x_type)) || !aligned(out, 2) || !aligned(workspace, 16))
    return MUA_ERR_ALIGN;
  const bool same = out == x && x_type == MUA_BF16 && out_row_stride == x_row_stride &&
                    (h->count == 1 || out_matrix_stride == x_matrix_stride);
  const int64_t x_span = last * x_matrix_stride + (h->rows - 1) * x_row_stride + row;
  const int64_t out_span = last * out_matrix_stride + (h->rows - 1) * out_row_stride + row;
  if (!same && overlap(x, x_span * type_size(x_type), out, out_span * 2)) return MUA_ERR_ARG;
  if (overlap(x, x_span * type_size(x_type), workspace, h->workspace_bytes) ||
      overlap(out, out_span * 2, workspace, h->workspace_bytes))
    return MUA_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const Target to = {false, out, MUA_BF16, out_matrix_stride, out_row_stride, 1.0, 0.0f};
  uint32_t* status = reinterpret_cast<uint32_t*>(ws) + mua::kMuonHdrStatus;
  if (h->small) {
    const mua::MuonView v = {const_cast<void*>(x), x_type, x_matrix_stride, x_row_stride};
    const cudaError_t e =
        mua::muon_launch_small(shape(h, h->count), iteration(h, 0, h->count, to, status), v,
                               eps, h->ex[0], st);
    return e == cudaSuccess ? MUA_OK : fail(e, "orthogonalization kernel launch");
  }
  double* partials = reinterpret_cast<double*>(ws + h->off_partials);
  for (int32_t first = 0; first < h->count; first += h->group) {
    const int32_t count = std::min(h->group, h->count - first);
    const mua::MuonView v = {
        static_cast<uint8_t*>(const_cast<void*>(x)) + first * x_matrix_stride * type_size(x_type),
        x_type, x_matrix_stride, x_row_stride};
    cudaError_t e = mua::muon_launch_norm(shape(h, count), v, partials, st);
    if (e != cudaSuccess) return fail(e, "norm kernel launch");
    e = mua::muon_launch_load(shape(h, count), v, partials, eps, h->ex[0], ws + h->off_x[0],
                              reinterpret_cast<float*>(ws + h->off_factor), counters(h, ws), st);
    if (e != cudaSuccess) return fail(e, "load kernel launch");
    const int rc = iterate(h, ws, first, count, to, status, st);
    if (rc != MUA_OK) return rc;
  }
  return MUA_OK;
}

int mua_muon_step(mua_muon_t h, void* params, int32_t params_type, const void* grads,
                  int32_t grads_type, void* state, void* workspace, float lr, float scale,
                  float beta, int32_t nesterov, float eps, float wd, int64_t t, uint64_t seed,
                  void* stream) {
  if (!h || !params || !grads || !state || !workspace) return MUA_ERR_ARG;
  if (!valid_type(params_type) || !valid_type(grads_type) || t < 1) return MUA_ERR_ARG;
  if (!finite_f(lr) || !finite_f(scale) || !finite_f(wd) || !finite_f(eps) || eps < 0.0f)
    return MUA_ERR_ARG;
  if (!(beta >= 0.0f && beta < 1.0f)) return MUA_ERR_ARG;
  if (!aligned(params, type_size(params_type)) || !aligned(grads, type_size(grads_type)) ||
      !aligned(state, 16) || !aligned(workspace, 16))
    return MUA_ERR_ALIGN;
  const int64_t ps = value_bytes(h, params_type), gs = value_bytes(h, grads_type);
  if (overlap(params, ps, grads, gs) || overlap(state, h->state_bytes, workspace, h->workspace_bytes) ||
      overlap(params, ps, state, h->state_bytes) || overlap(grads, gs, state, h->state_bytes) ||
      overlap(params, ps, workspace, h->workspace_bytes) ||
      overlap(grads, gs, workspace, h->workspace_bytes))
    return MUA_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int64_t n = (int64_t)h->rows * h->cols;
  const Target to = {true, params, params_type, n, h->cols,
                     (double)lr * (double)scale, (float)(1.0 - (double)lr * (double)wd)};
  uint32_t* status = static_cast<uint32_t*>(state) + mua::kMuonHdrStatus;
  if (h->small) {
    const cudaError_t e = mua::muon_launch_small_step(
        shape(h, h->count), iteration(h, 0, h->count, to, status), quant(h, state, 0), grads,
        grads_type, beta, nesterov != 0, random_keys(h, 0, t, seed), eps, h->ex[0], st);
    return e == cudaSuccess ? MUA_OK : fail(e, "step kernel launch");
  }
  double* partials = reinterpret_cast<double*>(ws + h->off_partials);
  float* factor = reinterpret_cast<float*>(ws + h->off_factor);
  for (int32_t first = 0; first < h->count; first += h->group) {
    const int32_t count = std::min(h->group, h->count - first);
    const mua::MuonShape s = shape(h, count);
    const mua::MuonQuant q = quant(h, state, first);
    const uint8_t* g = static_cast<const uint8_t*>(grads) + first * n * type_size(grads_type);
    cudaError_t e = mua::muon_launch_direction_norm(s, q, g, grads_type, beta, nesterov != 0,
                                                    partials, st);
    if (e != cudaSuccess) return fail(e, "direction norm kernel launch");
    e = mua::muon_launch_momentum(s, q, g, grads_type, beta, nesterov != 0,
                                  random_keys(h, first, t, seed), nullptr, 0, partials, eps,
                                  h->ex[0], ws + h->off_x[0], factor, counters(h, ws), st);
    if (e != cudaSuccess) return fail(e, "momentum kernel launch");
    const int rc = iterate(h, ws, first, count, to, status, st);
    if (rc != MUA_OK) return rc;
  }
  return MUA_OK;
}

int mua_muon_get_status(mua_muon_t h, const void* buffer, void* stream, int32_t* out) {
  if (!h || !buffer || !out) return MUA_ERR_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint32_t* hdr = static_cast<const uint32_t*>(buffer);
  cudaError_t e = cudaMemcpyAsync(out, hdr + mua::kMuonHdrStatus, 4, cudaMemcpyDeviceToHost, s);
  if (e != cudaSuccess) return fail(e, "status copy");
  e = cudaStreamSynchronize(s);
  return e == cudaSuccess ? MUA_OK : fail(e, "status synchronize");
}

const char* mua_muon_last_cuda_error(void) { return g_error; }

}  // extern "C"
