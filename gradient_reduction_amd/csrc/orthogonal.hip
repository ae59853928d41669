// Orthogonalising matrices by Newton-Schulz products, and the momentum update
// that uses it.  For every matrix G (rows x cols; m = the smaller side, n the
// larger, G transposed where rows > cols):
//   X <- U / (|U|_F + eps)              U = G, or the momentum's look-ahead
//   repeat: A = X XT; B = b A + c A A; X <- a X + B X
//   O = X, or W <- (1 - lr wd) W - lr s X
// Every product is one launch for a chunk of up to kNsChunk matrices: a workgroup
// finds its matrix by its tile number.  A and B are symmetric, so only tiles
// on and above their diagonal are computed and each is written twice.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "product.h"

namespace dc {
namespace {

constexpr int kNsChunk = 128;         // matrices whose products share launches
constexpr int kNsPart = 48;           // of them whose addresses fit one launch's arguments
// Planes of a chunk: the workspace does not grow with a model's layers.  A
// 7B-class layer takes 2.4 GiB in pairs and has 12 rounds of tiles a product.
constexpr int64_t kNsBytes = (int64_t)4 << 30;
constexpr int kNormParts = 256;       // partial sums of squares per matrix, at most
constexpr int64_t kNormSpan = 16384;  // elements per partial sum, at least

// What X, A and B are held in: one fp16 (11 bits), or two, a value and what it
// leaves (22 bits), multiplied as high high + high low + low high (three
// products of 16 bits take a fifth of one product of fp32 on these matrix
// cores).  Two leave about 1e-6 of |O|_F after five steps (0.5e-6 to 1.6e-6, single
// small matrices up to 2e-6); the same steps in fp32 leave 0.3e-6 to 3.6e-6.  One leaves 1.3e-3 to 1.6e-3 where the smaller
// side is kPairUnder or more, less than the rounding of O to bf16; on smaller
// matrices, whose few singular values do not average the roundings, it left 8e-3
// at worst, and there two cost little.  48 matrices of 1024 x 1024 to 4096 x 1024
// with their momenta and fp32 weights take 2.9 ms with one, 6.8 with two, and the
// weights are off by 3.2e-6 and 4.1e-8.
using Held = _Float16;
constexpr int32_t kPairUnder = 256;

// One matrix of a chunk.  Its planes in the workspace, in values from the
// planes' base: X [m][ldx], the next X [m][ldx], A [m][lda], B [m][lda]; with
// two values each is a pair of planes.
struct NsMatrix {
  const void* grad;
  void* out;
  float* momentum;
  int64_t ld_grad, ld_out;
  int64_t base;
  int32_t rows, cols;
  float scale;  // lr times the shape's factor (update only)
};

// Tables that travel as kernel arguments: up to kNsPart matrices with their
// addresses, or a whole chunk's planes.
struct NsTable {
  int32_t count;
  int32_t first;  // of the chunk
  NsMatrix m[kNsPart];
};

struct NsPlanes {
  int32_t count;
  struct {
    int64_t base;
    int32_t rows, cols;
  } m[kNsChunk];
};

// First tile of every matrix of a table, and their number.
struct NsTiles {
  int32_t begin[kNsChunk + 1];
};

static_assert(sizeof(NsTable) + sizeof(NsTiles) + 128 <= 4096, "kernel arguments");
static_assert(sizeof(NsPlanes) + sizeof(NsTiles) + 128 <= 4096, "kernel arguments");

__host__ __device__ inline int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }
__host__ __device__ inline int64_t up128(int64_t v) { return (v + 127) / 128 * 128; }

struct NsShape {
  int64_t m, n, ldx, lda, x_size, a_size;
  bool flip;  // X is G transposed
  __host__ __device__ NsShape(int64_t rows, int64_t cols) {
    flip = rows > cols;
    m = flip ? cols : rows;
    n = flip ? rows : cols;
    ldx = up8(n);
    lda = up8(m);
    x_size = up128(m * ldx);
    a_size = up128(m * lda);
  }
  __host__ __device__ int64_t values(int pair) const { return 2 * pair * (x_size + a_size); }
};

__host__ __device__ inline int32_t norm_parts(int64_t rows, int64_t cols) {
  const int64_t p = (rows * cols + kNormSpan - 1) / kNormSpan;
  return (int32_t)(p < 1 ? 1 : p > kNormParts ? kNormParts : p);
}

// The matrix of tile t: the last one whose first tile is at or before t.  Every
// lane looks at one or two.
__device__ __forceinline__ int find_matrix(const NsTiles& tiles, int count, int32_t t) {
  const int lane = threadIdx.x & 63;
  int n = __popcll(__ballot(lane < count && tiles.begin[lane] <= t));
  if (count > 64) n += __popcll(__ballot(lane + 64 < count && tiles.begin[lane + 64] <= t));
  return __builtin_amdgcn_readfirstlane(n - 1);
}

// This workgroup's tile of its matrix: one XCD's workgroups take a run of
// neighbouring tiles of every matrix.  (Runs over the whole list would give
// the matrices with the longest sums, which come first, to one XCD.)
__device__ __forceinline__ int32_t matrix_tile(const NsTiles& tiles, int e) {
  return (int32_t)xcd_run((int32_t)blockIdx.x - tiles.begin[e], tiles.begin[e + 1] - tiles.begin[e]);
}

struct NsUpdate {
  float mu, decay;   // decay = lr wd
  int32_t nesterov;
  const float* lr_scale;  // device, or null
};

// |U|_F^2 in parts, in fp64 (fp32 gradients of 1e-30 and 1e30 both have a
// square there), and the momentum's step: m <- mu m + g.  Bound by its bytes:
// 100 M elements of bf16 gradients and fp32 momenta, 1 GB, take 190 us.
template <class G, bool MOM>
__global__ void __launch_bounds__(256) k_ns_norm(NsTable tab, NsTiles tiles, NsUpdate up, double* parts) {
  const int e = find_matrix(tiles, tab.count, (int32_t)blockIdx.x);
  const NsMatrix& x = tab.m[e];
  const int part = (int)blockIdx.x - tiles.begin[e], np = tiles.begin[e + 1] - tiles.begin[e];
  const int64_t per_row = (x.cols + 3) / 4, groups = x.rows * per_row;
  const G* grad = static_cast<const G*>(x.grad);
  double s = 0;
  for (int64_t q = (int64_t)part * 256 + threadIdx.x; q < groups; q += (int64_t)np * 256) {
    int64_t r, c;
    if (groups < ((int64_t)1 << 31)) {
      r = (uint32_t)q / (uint32_t)per_row;
      c = ((uint32_t)q - (uint32_t)r * (uint32_t)per_row) * (int64_t)4;
    } else {
      r = q / per_row;
      c = (q - r * per_row) * 4;
    }
    const int n = (int)(x.cols - c < 4 ? x.cols - c : 4);
    f32x4 u = load_n<4>(grad + r * x.ld_grad + c, n);
    if constexpr (MOM) {
      float* mp = x.momentum + r * x.cols + c;
      const f32x4 g = u;
      u = load_n<4>(mp, n);
#pragma unroll
      for (int t = 0; t < 4; ++t) u[t] = fmaf(up.mu, u[t], g[t]);
      store_n<4>(mp, u, n);
      if (up.nesterov) {
#pragma unroll
        for (int t = 0; t < 4; ++t) u[t] = fmaf(up.mu, u[t], g[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) s = fma((double)u[t], (double)u[t], s);
  }
  __shared__ double sum[4];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_down(s, d);
  if ((threadIdx.x & 63) == 0) sum[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) parts[(int64_t)(tab.first + e) * kNormParts + part] = sum[0] + sum[1] + sum[2] + sum[3];
}

// N held values at `at` of a plane; the second plane of a pair lies `size`
// values on.  v is settled first: a multiplication that made it is otherwise
// folded into one of its two conversions (v_fma_mixlo_f16 rounds the product
// once, v_cvt_pk_f16_f32 the product's fp32), and the low half then belongs to
// another high half than the stored one.  That left up to 6e-5 of |O|_F
// instead of 1e-6.
template <int P, int N, class V>
__device__ __forceinline__ void store_held(Held* p, int64_t at, int64_t size, V v) {
#pragma unroll
  for (int t = 0; t < N; ++t) {
    float settled = v[t];
    asm("" : "+v"(settled));
    v[t] = settled;
  }
  store_n<N>(p + at, v, N);
  if constexpr (P == 2) {
#pragma unroll
    for (int t = 0; t < N; ++t) v[t] -= (float)(Held)v[t];
    store_n<N>(p + size + at, v, N);
  }
}

// X = U scale / (|U|_F + eps), transposed where rows > cols, 64 x 64 at a
// time; columns n .. ldx - 1 of X are zero.  Bound by its bytes: the same 100 M
// elements into pairs, 1 GB, take 214 us.
template <int P, class G, bool MOM>
__global__ void __launch_bounds__(256) k_ns_load(NsTable tab, NsTiles tiles, NsUpdate up, const double* parts,
                                                 float eps, float scale, Held* planes) {
  const int e = find_matrix(tiles, tab.count, (int32_t)blockIdx.x);
  const NsMatrix& x = tab.m[e];
  const NsShape sh(x.rows, x.cols);
  __shared__ float tile[64][65];
  __shared__ double total[4];
  const int np = norm_parts(x.rows, x.cols);
  double s = threadIdx.x < (unsigned)np ? parts[(int64_t)(tab.first + e) * kNormParts + threadIdx.x] : 0.0;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_down(s, d);
  if ((threadIdx.x & 63) == 0) total[threadIdx.x >> 6] = s;
  __syncthreads();
  // the factor and the product with it in fp64: neither leaves its range
  const double f = (double)scale / (sqrt(total[0] + total[1] + total[2] + total[3]) + (double)eps);
  const int32_t t = (int32_t)blockIdx.x - tiles.begin[e];
  const int32_t across = (x.cols + 63) / 64;
  const int64_t r0 = (int64_t)(t / across) * 64, c0 = (int64_t)(t % across) * 64;
  const G* grad = static_cast<const G*>(x.grad);
  const int c = (threadIdx.x & 15) * 4, l = threadIdx.x >> 4;
  Held* out = planes + x.base;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int rr = l + 16 * p;
    const int64_t r = r0 + rr, col = c0 + c;
    f32x4 u = {0.f, 0.f, 0.f, 0.f};
    if (r < x.rows && col < x.cols) {
      const int n = (int)(x.cols - col < 4 ? x.cols - col : 4);
      u = load_n<4>(grad + r * x.ld_grad + col, n);
      if constexpr (MOM) {
        const f32x4 g = u;
        u = load_n<4>(x.momentum + r * x.cols + col, n);
        if (up.nesterov) {
#pragma unroll
          for (int k = 0; k < 4; ++k) u[k] = fmaf(up.mu, u[k], g[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = (float)((double)u[k] * f);
    }
    if (!sh.flip) {
      if (r < sh.m && col < sh.ldx) store_held<P, 4>(out, r * sh.ldx + col, sh.x_size, u);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) tile[rr][c + k] = u[k];
    }
  }
  if (sh.flip) {
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int64_t i = c0 + l + 16 * p, j = r0 + c;  // X[i][j ..] = U[j ..][i]
      f32x4 u;
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = tile[c + k][l + 16 * p];
      if (i < sh.m && j < sh.ldx) store_held<P, 4>(out, i * sh.ldx + j, sh.x_size, u);
    }
  }
}

// The product of two operands that are pairs of planes, size_a and size_b
// apart; the small products first.  hook is called with the stages that hold
// B's own values (of each plane of it).
//
// An instruction rounds the sum it adds to four times (once for eight of its 32
// products), so a long sum collects roundings of its whole size: with A's sums
// in one piece 20 x 2000, 4000 x 24 and 48 x 4096 were off by 1.9e-6, 2.9e-6
// and 1.6e-6 of |O|_F, with sums of kFold stages that are added up apart (FOLD)
// by 1.4e-6, 1.5e-6 and 1.4e-6; one 1024 x 1024 matrix takes 284 us so, 278
// without.  (Most of the rest is that the eight products are cut off at 2^-24 of
// the largest.)  The other products' sums are as short as the smaller side: 308
// us with all of them so.  A 256 tile has no registers for it.
constexpr int kFold = 4;

// Up to kFew singular values do not average what is left out: their products
// of the low halves (2^-24 of a value, of one sign on A's diagonal) are taken
// too (64 tiles).  Without them 1 x 300 was off by 6.9e-7 of |O|_F and 4 x 1000
// by 1.3e-6, with them by 5.5e-7 and 9.8e-7; nine odd matrices, two of them
// with few, take 231.7 us so, 230.3 without.
constexpr int kFew = 64;

template <class Tile, int P, bool FOLD, class Acc, class Hook>
__device__ __forceinline__ void held_product(Operand<Held> a, int64_t size_a, Operand<Held> b, int64_t size_b,
                                             int64_t k, bool few, Acc& acc, Hook&& hook) {
  if constexpr (P == 2) {
    Operand<Held> low = a;
    low.p += size_a;
    if constexpr (Tile::MI * Tile::NI <= 4) {  // 64 tiles
      if (few) {
        Operand<Held> lows = b;
        lows.p += size_b;
        Tile::run(low, lows, 0, k, acc);
      }
    }
    Tile::run(low, b, 0, k, acc);
    low = b;
    low.p += size_b;
    Tile::run(a, low, 0, k, acc, hook);
  }
  if constexpr (P == 2 && FOLD) {
    f32x4 total[Tile::MI][Tile::NI] = {};
    auto fold = [&] {
#pragma unroll
      for (int i = 0; i < Tile::MI; ++i)
#pragma unroll
        for (int j = 0; j < Tile::NI; ++j) {
          total[i][j] += acc[i][j];
          acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    };
    fold();
    Tile::run(a, b, 0, k, acc, [&](LdsPtr la, int64_t k0) {
      hook(la, k0);
      if ((k0 / Tile::BK) % kFold == kFold - 1) fold();
    });
#pragma unroll
    for (int i = 0; i < Tile::MI; ++i)
#pragma unroll
      for (int j = 0; j < Tile::NI; ++j) acc[i][j] += total[i][j];
  } else {
    Tile::run(a, b, 0, k, acc, hook);
  }
}

// Tile t of the upper triangle of an nt x nt grid, by rows.
__device__ __forceinline__ void triangle_tile(int32_t t, int32_t nt, int32_t& ti, int32_t& tj) {
  int32_t row = 0, left = t;
  while (left >= nt - row) {
    left -= nt - row;
    ++row;
  }
  ti = row;
  tj = row + left;
}

// A = alpha X XT (POLY false: src = X, dst = A), or B = alpha (beta A + A A)
// (POLY true: src = A, dst = B; A is its own transpose).  Bound by the matrix
// cores: the four 4096 x 4096 and three 4096 x 11008 matrices of a 7B layer take
// 787 us for A and 484 us for B with one fp16, 1.12 and 1.05 PFLOP/s of the tiles
// that are computed, half of the whole product, and 2250 and 1410 us with pairs,
// 1.17 and 1.08; 952 tiles of 256 are 3.7 rounds.  One 1024 x 1024 matrix takes 10
// us each, 18 with pairs, a tile's latency.
template <int P, int BT, int WM, int WN, int S, bool POLY>
__global__ void __launch_bounds__(WM * WN * 64) k_ns_symmetric(NsPlanes tab, NsTiles tiles, Held* planes, int32_t next,
                                                               float alpha, float beta) {
  using Tile = TileProduct<Held, BT, BT, WM, WN, true, true, S>;
  const int e = find_matrix(tiles, tab.count, (int32_t)blockIdx.x);
  const int32_t t = matrix_tile(tiles, e);
  const NsShape sh(tab.m[e].rows, tab.m[e].cols);
  Held* x = planes + tab.m[e].base;
  Held* a_plane = x + 2 * P * sh.x_size;
  const Held* src = POLY ? a_plane : x + (next ? P * sh.x_size : 0);
  Held* dst = POLY ? a_plane + P * sh.a_size : a_plane;
  const int64_t ld = POLY ? sh.lda : sh.ldx, size = POLY ? sh.a_size : sh.x_size;
  int32_t ti, tj;
  triangle_tile(t, (int32_t)((sh.m + BT - 1) / BT), ti, tj);
  const int64_t i0 = (int64_t)ti * BT, j0 = (int64_t)tj * BT;
  const Operand<Held> a{src + i0 * ld, ld, (int32_t)(sh.m - i0 < BT ? sh.m - i0 : BT)};
  const Operand<Held> b{src + j0 * ld, ld, (int32_t)(sh.m - j0 < BT ? sh.m - j0 : BT)};
  f32x4 acc[Tile::MI][Tile::NI] = {};
  // B: beta A, its own transpose, comes into the sums from the stages that
  // hold it
  held_product<Tile, P, !POLY && BT <= 128>(a, size, b, size, ld, sh.m <= kFew, acc, [&](LdsPtr la, int64_t k) {
    if constexpr (POLY) Tile::add_b(la, k, i0, beta, acc);
  });
  // Columns m .. lda - 1 get zeros; the mirrored tile gets the same values.
  Tile::each(
      acc, true, ti != tj,
      [&](int i, int j, f32x8 v) {
        if (i >= a.rows || j0 + j >= sh.lda) return v;
        v *= alpha;
        store_held<P, 8>(dst, (i0 + i) * sh.lda + j0 + j, sh.a_size, v);
        return v;
      },
      [&](int j, int i, f32x8 v) {
        if (j < b.rows && i < a.rows) store_held<P, 8>(dst, (j0 + j) * sh.lda + i0 + i, sh.a_size, v);
      });
}

// X <- beta (a X + B X) into the other X plane, or out of it in the last step.
// The same 7B layer takes 1528 us with one fp16, 1.09 PFLOP/s, and 4430 with
// pairs, 1.12; 48 matrices of 1024 x 1024 to 4096 x 1024 in pairs 621 us, 0.99 (a
// tile's beginning and end are a fifth of its 48 stages), their last step with
// the weights 792 us.
enum : int { kNsNext = 0, kNsOut = 1, kNsWeight = 2 };

template <int P, class O, int BT, int WM, int WN, int S, int LAST, class Table>
__global__ void __launch_bounds__(WM * WN * 64) k_ns_step(Table tab, NsTiles tiles, Held* planes, int32_t next,
                                                          float a_coef, float beta, NsUpdate up) {
  using Tile = TileProduct<Held, BT, BT, WM, WN, true, false, S>;
  const int e = find_matrix(tiles, tab.count, (int32_t)blockIdx.x);
  const int32_t t = matrix_tile(tiles, e);
  const auto& x = tab.m[e];
  const NsShape sh(x.rows, x.cols);
  const Held* src = planes + x.base + (next ? P * sh.x_size : 0);
  Held* dst = planes + x.base + (next ? 0 : P * sh.x_size);
  const Held* poly = planes + x.base + 2 * P * sh.x_size + P * sh.a_size;
  int64_t ti, tj;
  band_tile(t, (sh.m + BT - 1) / BT, (sh.n + BT - 1) / BT, 8, ti, tj);
  const int64_t i0 = ti * BT, j0 = tj * BT;
  const Operand<Held> a{poly + i0 * sh.lda, sh.lda, (int32_t)(sh.m - i0 < BT ? sh.m - i0 : BT)};
  const Operand<Held> b{src + j0, sh.ldx, (int32_t)(sh.ldx - j0 < BT ? sh.ldx - j0 : BT)};
  f32x4 acc[Tile::MI][Tile::NI] = {};
  // a X comes into the sums from the stages that hold it: with the tile read
  // again after the sums, every unit waited for memory at once
  held_product<Tile, P, false>(a, sh.a_size, b, sh.x_size, sh.m, sh.m <= kFew, acc,
                        [&](LdsPtr la, int64_t k) { Tile::add_b(la, k, i0, a_coef, acc); });
  O* out = nullptr;
  int64_t ld_out = 0;
  float scale = 1.f, keep = 1.f;
  if constexpr (LAST != kNsNext) {
    out = static_cast<O*>(x.out);
    ld_out = x.ld_out;
    const float rate = LAST == kNsWeight && up.lr_scale ? *up.lr_scale : 1.f;
    scale = x.scale * rate;
    keep = 1.f - up.decay * rate;
  }
  auto write = [&](O* p, f32x8 v, int64_t n) {
    if constexpr (LAST == kNsWeight) v = keep * load_n<8>(p, n) - scale * v;
    store_n<8>(p, v, n);
  };
  const bool flip = LAST != kNsNext && sh.flip;
  Tile::each(
      acc, !flip, flip,
      [&](int i, int j, f32x8 v) {
        if (i >= a.rows || j >= b.rows) return v;
        v *= beta;
        if constexpr (LAST == kNsNext) store_held<P, 8>(dst, (i0 + i) * sh.ldx + j0 + j, sh.x_size, v);
        else write(out + (i0 + i) * ld_out + j0 + j, v, sh.n - (j0 + j));
        return v;
      },
      [&](int j, int i, f32x8 v) {
        if (j0 + j >= sh.n || i >= a.rows) return;
        const int64_t n = a.rows - i;
        v *= beta;
        write(out + (j0 + j) * ld_out + i0 + i, v, n);
      });
}

// Largest |a x + b x^3 + c x^5| for 0 <= x <= top: at the ends or where the
// slope a + 3 b t + 5 c t^2 (t = x^2) is zero.
double step_top(const float* co, double top) {
  const double a = co[0], b = co[1], c = co[2];
  auto p = [&](double x) { return std::fabs(x * (a + x * x * (b + x * x * c))); };
  double best = p(top);
  double roots[2];
  int n = 0;
  if (c != 0) {
    const double d = 9 * b * b - 20 * a * c;
    if (d >= 0) {
      roots[n++] = (-3 * b + std::sqrt(d)) / (10 * c);
      roots[n++] = (-3 * b - std::sqrt(d)) / (10 * c);
    }
  } else if (b != 0) {
    roots[n++] = -a / (3 * b);
  }
  for (int k = 0; k < n; ++k)
    if (roots[k] > 0 && roots[k] < top * top) best = std::max(best, p(std::sqrt(roots[k])));
  return best;
}

// The powers of two by which X, A and B are held.  The largest singular value
// bounds every element: X0 has at most |X0|_F <= 1, each step's is bounded by
// its polynomial (with a thousandth for what is held having been rounded),
// |A| by the square, |B| by |b| A + |c| A A.  In fp16 the bound is held at
// 2^13 to 2^14, a quarter of the type's largest value; values down to 2^-27 of
// it keep all 11 bits.
constexpr double kSlack = 1.001;

struct NsScales {
  float x = 1.f, a = 1.f;
  float b[DC_NS_MAX_STEPS];
};

NsScales ns_scales(int32_t steps, const float* coeffs) {
  NsScales s;
  double top[DC_NS_MAX_STEPS + 1], most = kSlack;
  top[0] = kSlack;
  for (int k = 0; k < steps; ++k) {
    top[k + 1] = kSlack * step_top(coeffs + 3 * k, top[k]);
    most = std::max(most, top[k + 1]);
  }
  auto hold = [](double bound) { return (float)std::ldexp(1.0, 14 - std::max(-40, std::ilogb(bound) + 1)); };
  s.x = hold(most);
  s.a = hold(most * most);
  for (int k = 0; k < steps; ++k) {
    const double q = top[k] * top[k];
    s.b[k] = hold(std::max(1e-6, std::fabs(coeffs[3 * k + 1]) * q + std::fabs(coeffs[3 * k + 2]) * q * q));
  }
  return s;
}

// How many values hold one of a matrix's.
struct Holding {
  int32_t dtype, out_dtype, hold;
  int values(const dc_matrix& m) const {
    if (hold != DC_HOLD_AUTO) return hold == DC_HOLD_PAIR ? 2 : 1;
    return dtype == DC_F32 || out_dtype == DC_F32 || std::min(m.rows, m.cols) < kPairUnder ? 2 : 1;
  }
};

// f(pair, indices, count) for every chunk: matrices held alike, kNsChunk of
// them at most, and of 2^22 64 x 64 tiles (a grid holds 2^24) and kNsBytes of
// planes together unless it is one, in chunks of about one size.
template <class F>
void each_chunk(const Holding& held, const dc_matrix* mats, int32_t num, F&& f) {
  for (const int pair : {1, 2}) {
    int32_t left = 0;
    for (int32_t k = 0; k < num; ++k) left += held.values(mats[k]) == pair;
    for (int32_t k = 0; left > 0;) {
      const int32_t chunks = (left + kNsChunk - 1) / kNsChunk, most = (left + chunks - 1) / chunks;
      int32_t at[kNsChunk], count = 0;
      int64_t tiles = 0, bytes = 0;
      for (; k < num && count < most; ++k) {
        if (held.values(mats[k]) != pair) continue;
        tiles += ((int64_t)(mats[k].rows + 63) / 64) * ((mats[k].cols + 63) / 64);
        bytes += NsShape(mats[k].rows, mats[k].cols).values(pair) * (int64_t)sizeof(Held);
        if (count > 0 && (tiles > ((int64_t)1 << 22) || bytes > kNsBytes)) break;
        at[count++] = k;
      }
      f(pair, at, count);
      left -= count;
    }
  }
}

constexpr int64_t kPartsBytes = (int64_t)kNsChunk * kNormParts * 8;

template <class Table, class F>
int32_t fill_tiles(NsTiles& tiles, const Table& tab, F&& count) {
  int64_t t = 0;
  for (int k = 0; k < tab.count; ++k) {
    tiles.begin[k] = (int32_t)t;
    t += count(NsShape(tab.m[k].rows, tab.m[k].cols));
  }
  for (int k = tab.count; k <= kNsChunk; ++k) tiles.begin[k] = (int32_t)t;
  return (int32_t)t;
}

// The products of a step.
enum Product : int { kGram, kPoly, kStep };

// The tile (256, 128 or 64 square) that is estimated to take a product of the
// whole chunk fastest.  A compute unit takes stage_us for each stage and
// tile_us for a tile's beginning and end; tiles of one length run in whole
// rounds, of several lengths in the longest one's time or everybody's share
// and half a shortest one.
int ns_tile(const NsPlanes& tab, Product p, int pair) {
  int best = 0;
  double least = 0;
  for (const int tile : {256, 128, 64}) {
    const double tile_us = tile == 256 ? 6.0 : tile == 128 ? 1.5 : 0.5;
    double total = 0, count = 0, longest = 0, shortest = 1e30;
    for (int k = 0; k < tab.count; ++k) {
      const NsShape s(tab.m[k].rows, tab.m[k].cols);
      const double tm = (double)((s.m + tile - 1) / tile), tn = (double)((s.n + tile - 1) / tile);
      const double stages = std::ceil((p == kGram ? s.ldx : s.lda) / 64.0) * (pair == 2 ? 3 : 1);
      const double us = stages * stage_us(false, tile) + tile_us;
      const double tiles = p == kStep ? tm * tn : tm * (tm + 1) / 2;
      total += tiles * us;
      count += tiles;
      longest = std::max(longest, us);
      shortest = std::min(shortest, us);
    }
    const double us = shortest == longest ? std::ceil(count / kComputeUnits) * longest
                                          : std::max(longest, total / kComputeUnits + shortest / 2);
    if (best == 0 || us < least) {
      least = us;
      best = tile;
    }
  }
  return best;
}

// The tiles of a chunk's products.
struct NsCut {
  int gram, poly, step, last;
};

NsCut ns_cut(const NsPlanes& tab, int pair, bool update) {
  NsCut c{ns_tile(tab, kGram, pair), ns_tile(tab, kPoly, pair), ns_tile(tab, kStep, pair), 0};
  // The last step of an update also reads and writes the weights: two 128
  // tiles in a compute unit overlap that with products (40 matrices of 1024 x
  // 1024 and 4096 x 1024, fp32 weights: 295 us against 356 us of one 256 tile).
  c.last = update && c.step == 256 ? 128 : c.step;
  return c;
}

// The first tiles of a product's launch; returns their number.
template <class Table>
int32_t product_tiles(NsTiles& tiles, const Table& tab, Product p, int tile) {
  return fill_tiles(tiles, tab, [&](const NsShape& s) {
    const int64_t tm = (s.m + tile - 1) / tile, tn = (s.n + tile - 1) / tile;
    return p == kStep ? tm * tn : tm * (tm + 1) / 2;
  });
}

template <int P, bool POLY>
void launch_symmetric(const NsPlanes& tab, const NsTiles& tiles, int32_t n, int tile, Held* planes, int32_t next,
                      float alpha, float beta, hipStream_t stream) {
  auto launch = [&](auto kernel, int threads) {
    kernel<<<n, threads, 0, stream>>>(tab, tiles, planes, next, alpha, beta);
  };
  const bool deep = launch_stages(tile, n) == 4;
  if (tile == 256) launch(k_ns_symmetric<P, 256, 4, 2, 2, POLY>, 512);
  else if (tile == 128 && deep) launch(k_ns_symmetric<P, 128, 2, 4, 4, POLY>, 512);
  else if (tile == 128) launch(k_ns_symmetric<P, 128, 2, 4, 2, POLY>, 512);
  else launch(k_ns_symmetric<P, 64, 2, 2, 3, POLY>, 256);
}

template <int P, class O, int LAST, class Table>
void launch_step(const Table& tab, const NsTiles& tiles, int32_t n, int tile, Held* planes, int32_t next,
                 float a_coef, float beta, const NsUpdate& up, hipStream_t stream) {
  auto launch = [&](auto kernel, int threads) {
    kernel<<<n, threads, 0, stream>>>(tab, tiles, planes, next, a_coef, beta, up);
  };
  const bool deep = launch_stages(tile, n) == 4;
  if (tile == 256) launch(k_ns_step<P, O, 256, 4, 2, 2, LAST, Table>, 512);
  else if (tile == 128 && deep) launch(k_ns_step<P, O, 128, 2, 4, 4, LAST, Table>, 512);
  else if (tile == 128) launch(k_ns_step<P, O, 128, 2, 4, 2, LAST, Table>, 512);
  else launch(k_ns_step<P, O, 64, 2, 2, 3, LAST, Table>, 256);
}

// One chunk: `mats` in the order of their sums' lengths.
template <int P, class G, class O, bool MOM>
void ns_chunk(const NsMatrix* mats, int32_t count, const NsLaunch& a, const NsScales& sc, const NsUpdate& up,
              double* parts, Held* planes, hipStream_t stream) {
  // f(table of up to kNsPart matrices) over the chunk
  auto by_part = [&](auto f) {
    for (int32_t first = 0; first < count; first += kNsPart) {
      NsTable tab;
      tab.first = first;
      tab.count = std::min(kNsPart, count - first);
      std::copy(mats + first, mats + first + tab.count, tab.m);
      f(tab);
    }
  };
  by_part([&](const NsTable& tab) {
    NsTiles tiles;
    int32_t n = 0;
    for (int32_t k = 0; k < tab.count; n += norm_parts(tab.m[k].rows, tab.m[k].cols), ++k) tiles.begin[k] = n;
    for (int32_t k = tab.count; k <= kNsChunk; ++k) tiles.begin[k] = n;
    k_ns_norm<G, MOM><<<n, 256, 0, stream>>>(tab, tiles, up, parts);
  });
  by_part([&](const NsTable& tab) {
    NsTiles tiles;
    const int32_t n = fill_tiles(tiles, tab, [](const NsShape& s) { return ((s.m + 63) / 64) * ((s.n + 63) / 64); });
    k_ns_load<P, G, MOM><<<n, 256, 0, stream>>>(tab, tiles, up, parts, a.eps, sc.x, planes);
  });
  NsPlanes all;
  all.count = count;
  for (int32_t k = 0; k < count; ++k) all.m[k] = {mats[k].base, mats[k].rows, mats[k].cols};
  const NsCut cut = ns_cut(all, P, MOM);
  NsTiles gram, poly, step;
  const int32_t n_gram = product_tiles(gram, all, kGram, cut.gram), n_poly = product_tiles(poly, all, kPoly, cut.poly),
                n_step = product_tiles(step, all, kStep, cut.step);
  for (int32_t k = 0; k < a.steps; ++k) {
    const float ca = a.coeffs[3 * k], cb = a.coeffs[3 * k + 1], cc = a.coeffs[3 * k + 2];
    const int32_t next = k & 1;
    launch_symmetric<P, false>(all, gram, n_gram, cut.gram, planes, next, sc.a / (sc.x * sc.x), 0.f, stream);
    // B = c (A A + b / c A): a c too small for fp32 to see beside b stands for
    // zero
    const double c = std::fabs(cc) < std::fabs(cb) * 0x1p-30 ? std::fabs(cb) * 0x1p-30 : cc;
    launch_symmetric<P, true>(all, poly, n_poly, cut.poly, planes, next, (float)(c * sc.b[k] / ((double)sc.a * sc.a)),
                              c != 0 ? (float)(cb * sc.a / c) : 0.f, stream);
    if (k + 1 < a.steps) {
      launch_step<P, O, kNsNext>(all, step, n_step, cut.step, planes, next, ca * sc.b[k], 1.f / sc.b[k], up, stream);
    } else {
      by_part([&](const NsTable& tab) {
        NsTiles last;
        const int32_t n = product_tiles(last, tab, kStep, cut.last);
        launch_step<P, O, MOM ? kNsWeight : kNsOut>(tab, last, n, cut.last, planes, next, ca * sc.b[k],
                                                    1.f / (sc.b[k] * sc.x), up, stream);
      });
    }
  }
}

// A chunk's matrices, the longest sums first, so that short ones fill what they
// leave.
void sort_chunk(NsMatrix* mats, int32_t count) {
  std::sort(mats, mats + count, [](const NsMatrix& x, const NsMatrix& y) {
    return std::max(x.rows, x.cols) > std::max(y.rows, y.cols);
  });
}

template <class G, class O, bool MOM>
hipError_t ns_run(const NsLaunch& a, hipStream_t stream) {
  const NsScales sc = ns_scales(a.steps, a.coeffs);
  double* parts = static_cast<double*>(a.workspace);
  Held* planes = reinterpret_cast<Held*>(static_cast<char*>(a.workspace) + kPartsBytes);
  const NsUpdate up{a.mu, a.lr * a.weight_decay, a.nesterov, a.lr_scale};
  hipError_t status = hipSuccess;
  each_chunk(Holding{a.dtype, a.out_dtype, a.hold}, a.mats, a.num, [&](int pair, const int32_t* at, int32_t count) {
    if (status != hipSuccess) return;
    NsMatrix mats[kNsChunk];
    int64_t base = 0;
    for (int32_t k = 0; k < count; ++k) {
      const dc_matrix& d = a.mats[at[k]];
      mats[k] = NsMatrix{d.grad, d.out, d.momentum, d.ld_grad, d.ld_out, base, d.rows, d.cols,
                         a.lr * ns_factor(a.scale_mode, d.rows, d.cols)};
      base += NsShape(d.rows, d.cols).values(pair);
    }
    sort_chunk(mats, count);
    if (pair == 2) ns_chunk<2, G, O, MOM>(mats, count, a, sc, up, parts, planes, stream);
    else ns_chunk<1, G, O, MOM>(mats, count, a, sc, up, parts, planes, stream);
    status = hipGetLastError();
  });
  return status;
}

}  // namespace

float ns_factor(int32_t scale_mode, int32_t rows, int32_t cols) {
  if (scale_mode == DC_SCALE_ASPECT) return std::sqrt(std::max(1.f, (float)rows / (float)cols));
  if (scale_mode == DC_SCALE_RMS) return 0.2f * std::sqrt((float)std::max(rows, cols));
  return 1.f;
}

double ns_largest(int32_t steps, const float* coeffs) {
  double top = kSlack, most = top;
  for (int k = 0; k < steps; ++k) most = std::max(most, top = kSlack * step_top(coeffs + 3 * k, top));
  return most;
}

int64_t ns_workspace(int32_t dtype, int32_t out_dtype, int32_t hold, const dc_matrix* mats, int32_t num) {
  int64_t most = 0;
  each_chunk(Holding{dtype, out_dtype, hold}, mats, num, [&](int pair, const int32_t* at, int32_t count) {
    int64_t v = 0;
    for (int32_t k = 0; k < count; ++k) v += NsShape(mats[at[k]].rows, mats[at[k]].cols).values(pair);
    most = std::max(most, v);
  });
  return num ? kPartsBytes + most * (int64_t)sizeof(Held) : 0;
}

void ns_forms(int32_t dtype, int32_t out_dtype, int32_t hold, const dc_matrix* mats, int32_t num, bool update,
              int32_t index, LaunchForm forms[4]) {
  each_chunk(Holding{dtype, out_dtype, hold}, mats, num, [&](int pair, const int32_t* at, int32_t count) {
    const int32_t* own = std::find(at, at + count, index);
    if (own == at + count) return;
    NsMatrix sorted[kNsChunk];
    for (int32_t k = 0; k < count; ++k) {
      sorted[k] = NsMatrix{};
      sorted[k].rows = mats[at[k]].rows;
      sorted[k].cols = mats[at[k]].cols;
    }
    sort_chunk(sorted, count);
    NsPlanes all;
    all.count = count;
    for (int32_t k = 0; k < count; ++k) all.m[k] = {0, sorted[k].rows, sorted[k].cols};
    const NsCut cut = ns_cut(all, pair, update);
    NsTiles tiles;
    auto form = [&](Product p, int tile) {
      return LaunchForm{tile, launch_stages(tile, product_tiles(tiles, all, p, tile)), 1};
    };
    forms[0] = form(kGram, cut.gram);
    forms[1] = form(kPoly, cut.poly);
    forms[2] = form(kStep, cut.step);
    // the last step goes by parts of kNsPart matrices
    const dc_matrix& m = mats[*own];
    int32_t k = 0;
    while (sorted[k].rows != m.rows || sorted[k].cols != m.cols) ++k;
    NsPlanes part;
    part.count = std::min(kNsPart, count - k / kNsPart * kNsPart);
    std::copy(all.m + k / kNsPart * kNsPart, all.m + k / kNsPart * kNsPart + part.count, part.m);
    forms[3] = LaunchForm{cut.last, launch_stages(cut.last, product_tiles(tiles, part, kStep, cut.last)), 1};
  });
}

hipError_t launch_ns(const NsLaunch& a, hipStream_t stream) {
  if (a.num == 0) return hipSuccess;
  if (!a.update) {
    if (a.dtype == DC_F32) return ns_run<float, float, false>(a, stream);
    return ns_run<__bf16, __bf16, false>(a, stream);
  }
  if (a.dtype == DC_F32) {
    if (a.out_dtype == DC_F32) return ns_run<float, float, true>(a, stream);
    return ns_run<float, __bf16, true>(a, stream);
  }
  if (a.out_dtype == DC_F32) return ns_run<__bf16, float, true>(a, stream);
  return ns_run<__bf16, __bf16, true>(a, stream);
}

}  // namespace dc
