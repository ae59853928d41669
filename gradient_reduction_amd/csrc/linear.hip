// The linear layer's kernels: forward product with bias, activation and
// residual in its epilogue, the bias-and-activation backward, and the two
// backward products.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"
#include "product.h"

namespace dc {
namespace {

// Activations and their slopes in fp32 from the hardware's 2^x and 1/x:
// activations to 2^-22 of the larger of argument and result, slopes to 2^-20
// (over -15 .. 15).  GELU's negative tail is off by about 2^-20 of itself at -5,
// 2^-19 at -9 and 2^-18 at -13, from the rounding of v^2; slopes have no such
// bound near their zeros.  With the library's exp, erfc and correctly
// rounded division the elementwise backward was bound by its arithmetic (129
// us on 8192 x 11008 bf16 where its bytes take 84).

// exp(x), x taken into [-150, 88] (zero from -104 on; outside, what the
// product rounds off would be infinite less infinite): 2^(x log2 e) with what
// the product rounds off.
__device__ __forceinline__ float exp_fast(float x) {
  x = __builtin_amdgcn_fmed3f(x, -150.f, 88.f);
  const float t = x * 1.44269504f;
  const float r = fmaf(x, 1.44269504f, -t) + x * 1.92596299e-8f;
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, r * 0.693147181f, e);
}

// 1 / (1 + exp(-v)); under -87 zero, so that a v of any size times it is
// within 2e-36 of its limit.
__device__ __forceinline__ float sigmoid(float v) {
  return v < -87.f ? 0.f : __builtin_amdgcn_rcpf(1.f + exp_fast(-v));
}

// Phi(v), the normal distribution's, and e = exp(-v^2 / 2).  With z = |v| /
// sqrt 2 and t = 1 / (1 + z / 2), erfc(z) exp(z^2) / t is a smooth function of
// t on (0, 1]: the polynomial is its least-squares fit in relative error,
// reweighted towards the least maximum (4e-8 over z < 9.5, 4e-7 as computed
// here); past that e is zero in fp32.
__device__ __forceinline__ float normal_cdf(float v, float& e) {
  e = exp_fast(-0.5f * v * v);
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(v), 0.353553391f, 1.f));
  float p = -5.889142478e-02f;
  p = fmaf(p, t, 2.837050295e-01f);
  p = fmaf(p, t, -4.853898047e-01f);
  p = fmaf(p, t, 2.759848175e-01f);
  p = fmaf(p, t, -2.518203246e-02f);
  p = fmaf(p, t, 2.020715627e-01f);
  p = fmaf(p, t, 2.432606008e-01f);
  p = fmaf(p, t, 2.823535357e-01f);
  p = fmaf(p, t, 2.820876737e-01f);
  const float tail = 0.5f * e * p * t;
  return v < 0.f ? tail : 1.f - tail;
}

__device__ __forceinline__ float activate(float v, int act) {
  float e;
  switch (act) {
    case DC_ACT_RELU: return v > 0.f || v != v ? v : 0.f;
    case DC_ACT_GELU: return v * normal_cdf(v, e);
    case DC_ACT_SILU: return v * sigmoid(v);
    default: return v;
  }
}

__device__ __forceinline__ float activation_slope(float v, int act) {
  switch (act) {
    case DC_ACT_RELU: return v > 0.f ? 1.f : 0.f;
    case DC_ACT_GELU: {
      float e;
      const float phi = normal_cdf(v, e);
      return fmaf(0.39894228040143268f * v, e, phi);
    }
    case DC_ACT_SILU: {
      const float p = sigmoid(v);
      return p * fmaf(v, 1.f - p, 1.f);
    }
    default: return 1.f;
  }
}

// What happens to the sums v of columns j .. of row i.
template <class T>
struct LinearEpilogue {  // y = act(v + bias) + residual, pre = v + bias
  LinearOut o;
  int64_t n_cols;
  template <class V>
  __device__ void operator()(int64_t i, int64_t j, V v) const {
    constexpr int N = sizeof(V) / 4;
    const int64_t n = n_cols - j;
    if (o.bias) v += load_n<N>(static_cast<const T*>(o.bias) + j, n);
    if (o.pre) store_n<N>(static_cast<T*>(o.pre) + i * o.ld_pre + j, v, n);
    if (o.act != DC_ACT_NONE) {
#pragma unroll
      for (int t = 0; t < N; ++t) v[t] = activate(v[t], o.act);
    }
    if (o.residual) v += load_n<N>(static_cast<const T*>(o.residual) + i * o.ld_res + j, n);
    store_n<N>(static_cast<T*>(o.out) + i * o.ld_out + j, v, n);
  }
};

template <class G>
struct GradEpilogue {  // out = (accumulate ? out : 0) + v
  LinearOut o;
  int64_t n_cols;
  template <class V>
  __device__ void operator()(int64_t i, int64_t j, V v) const {
    constexpr int N = sizeof(V) / 4;
    G* p = static_cast<G*>(o.out) + i * o.ld_out + j;
    if (o.accumulate) v += load_n<N>(p, n_cols - j);
    store_n<N>(p, v, n_cols - j);
  }
};

struct ProductArgs {
  const void *a, *b;
  int64_t ld_a, ld_b;
  int64_t m, n, k;
  int64_t tiles_m, tiles_n;
  int32_t splits;
  int64_t k_per_split;  // a multiple of the stage depth
  float* partial;       // [splits][m][ld_partial] when splits > 1
  int64_t ld_partial;
};

// One tile of C = A B (product.h) and its epilogue; y = x wT, dx = dz w and dw
// = dzT x are its three kinds.  Bound by the matrix cores where the tiles fill
// the chip: 8192 x 11008 over 4096 bf16 takes 690 to 715 us with silu and pre
// kept (1.05 PFLOP/s), dx 565 (1.31) and dw added to fp32 680 (1.09: 688 tiles of
// 256 are 2.7 rounds over the units, paid as 3), the first calls after idling a
// quarter more.  Tiles are walked in bands
// of eight rows, one XCD's workgroups on neighbours, so that an L2 serves what
// they share.  Odd fp32 rows go through registers: 777 x 1003 over 515 takes
// 23 us, bound by the latency of a tile's 17 stages.
template <class T, int BM, int BN, int WM, int WN, bool KCA, bool KCB, int S, class Epi>
__global__ void __launch_bounds__(WM * WN * 64) k_product(ProductArgs g, Epi epi) {
  using P = TileProduct<T, BM, BN, WM, WN, KCA, KCB, S>;
  const int64_t per = g.tiles_m * g.tiles_n;
  const int64_t t = xcd_run(blockIdx.x, gridDim.x);
  const int32_t split = (int32_t)(t / per);
  int64_t ti, tj;
  band_tile(t - split * per, g.tiles_m, g.tiles_n, 8, ti, tj);
  const int64_t i0 = ti * BM, j0 = tj * BN;
  Operand<T> a{static_cast<const T*>(g.a) + (KCA ? i0 * g.ld_a : i0), g.ld_a,
               (int32_t)(g.m - i0 < BM ? g.m - i0 : BM)};
  Operand<T> b{static_cast<const T*>(g.b) + (KCB ? j0 * g.ld_b : j0), g.ld_b,
               (int32_t)(g.n - j0 < BN ? g.n - j0 : BN)};
  const int64_t k0 = split * g.k_per_split;
  const int64_t k1 = k0 + g.k_per_split < g.k ? k0 + g.k_per_split : g.k;
  f32x4 acc[P::MI][P::NI] = {};
  P::run(a, b, k0, k1, acc);
  float* part = g.splits > 1 ? g.partial + split * g.m * g.ld_partial : nullptr;
  P::each(
      acc, true, false,
      [&](int i, int j, f32x8 v) {
        if (i >= a.rows || j >= b.rows) return v;
        if (part) store_n<8>(part + (i0 + i) * g.ld_partial + j0 + j, v, 8);
        else epi(i0 + i, j0 + j, v);
        return v;
      },
      [](int, int, f32x8) {});
}

// The splits of a long k added in their order, then the epilogue.
template <class Epi>
__global__ void __launch_bounds__(256) k_product_join(const float* partial, int64_t ld, int32_t splits, int64_t m,
                                                      int64_t n, Epi epi) {
  const int64_t groups = (n + 3) / 4;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= m * groups) return;
  const int64_t i = at / groups, j = (at - i * groups) * 4;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int32_t s = 0; s < splits; ++s)
    v += *reinterpret_cast<const f32x4*>(partial + ((int64_t)s * m + i) * ld + j);
  epi(i, j, v);
}

// How a product of m x n over k is cut: the tile (256, 128 or 64 square) and
// the splits of k whose estimated time is least.
struct Cut {
  int32_t tile, splits;
  int64_t k_per_split, ld_partial;
  int64_t partial_bytes(int64_t m) const { return splits > 1 ? splits * m * ld_partial * 4 : 0; }
};

Cut cut(int32_t dtype, int64_t m, int64_t n, int64_t k) {
  const bool f32 = dtype == DC_F32;
  const int64_t bk = f32 ? 32 : 64;
  // A stage alone in its compute unit takes `alone` at least (its loads'
  // latency; fp32's matrix instructions hide less of it), and `held`
  // workgroups of a tile share a unit.
  const double alone = f32 ? 0.6 : 0.4;
  const int64_t stages = std::max<int64_t>(1, (k + bk - 1) / bk);
  Cut best{};
  double least = 0;
  for (const int32_t tile : {256, 128, 64}) {
    const double held = tile == 256 ? 1 : tile == 128 ? 2 : 3, busy = stage_us(f32, tile);
    const int64_t tiles = std::max<int64_t>(1, ((m + tile - 1) / tile) * ((n + tile - 1) / tile));
    for (int64_t want = 1; want <= 64; ++want) {
      if (want > 1 && (want > stages / 4 || tiles * want > 4 * kComputeUnits)) break;
      const int64_t per = (stages + want - 1) / want, splits = (stages + per - 1) / per;
      const double a_unit = (double)((tiles * splits + kComputeUnits - 1) / kComputeUnits);
      const double full = std::floor(a_unit / held), rest = a_unit - full * held;
      double us = per * (full * std::max(alone, held * busy) + (rest > 0 ? std::max(alone, rest * busy) : 0.0));
      // the sums written and read again, and a launch more
      if (splits > 1) us += 3.0 + splits * m * n * 8.0 / 4e6;
      if (best.tile == 0 || us < least) {
        least = us;
        best = Cut{tile, (int32_t)splits, per * bk, (n + 7) / 8 * 8};
      }
    }
  }
  return best;
}

template <class T, int BT, int WM, int WN, int S, bool KCA, bool KCB, class Epi>
void launch_product(const ProductArgs& g, bool direct, const Epi& epi, hipStream_t stream) {
  const dim3 grid((uint32_t)(g.tiles_m * g.tiles_n * g.splits));
  if (direct) k_product<T, BT, BT, WM, WN, KCA, KCB, S, Epi><<<grid, WM * WN * 64, 0, stream>>>(g, epi);
  else k_product<T, BT, BT, WM, WN, KCA, KCB, 1, Epi><<<grid, WM * WN * 64, 0, stream>>>(g, epi);
}

template <class T, bool KCA, bool KCB, class Epi>
hipError_t product(int32_t dtype, const void* a, int64_t ld_a, const void* b, int64_t ld_b, int64_t m, int64_t n,
                   int64_t k, float* partial, const Epi& epi, hipStream_t stream) {
  const Cut c = cut(dtype, m, n, k);
  const ProductArgs g{a, b, ld_a, ld_b, m, n, k, (m + c.tile - 1) / c.tile, (n + c.tile - 1) / c.tile, c.splits,
                      c.k_per_split, partial, c.ld_partial};
  const bool direct = direct_operand<T>(a, ld_a, KCA ? k : m) && direct_operand<T>(b, ld_b, KCB ? k : n);
  const int32_t stages = launch_stages(c.tile, g.tiles_m * g.tiles_n * g.splits);
  if (c.tile == 256) launch_product<T, 256, 4, 2, 2, KCA, KCB>(g, direct, epi, stream);
  else if (c.tile == 128 && stages == 4) launch_product<T, 128, 2, 4, 4, KCA, KCB>(g, direct, epi, stream);
  else if (c.tile == 128) launch_product<T, 128, 2, 4, 2, KCA, KCB>(g, direct, epi, stream);
  else launch_product<T, 64, 2, 2, 3, KCA, KCB>(g, direct, epi, stream);
  if (c.splits > 1) {
    const int64_t groups = m * ((n + 3) / 4);
    k_product_join<Epi><<<dim3((uint32_t)((groups + 255) / 256)), 256, 0, stream>>>(partial, c.ld_partial, c.splits,
                                                                                  m, n, epi);
  }
  return hipGetLastError();
}

// A few rows (a single token's, or a decoding batch's): x wT with w streamed
// once from memory straight into the matrix cores' layout, no LDS between.  A
// workgroup takes 16 NI outputs and its eight waves k's groups in turn, so that
// enough loads are in flight and what is being read of a row is one run; their
// sums are added in the waves' order.  Bound by w's bytes and, from about eight
// rows on, by what a compute unit can fetch, which x shares: 16 x 4096 x 11008
// bf16 takes 22 us, 17 with x left out, and more loads in flight, 16 waves or
// 32 outputs a workgroup take 24, 24 and 33.
template <class T, int TI, int NI, bool DIRECT, class Epi>
__global__ void __launch_bounds__(512) k_linear_few(const T* x, int64_t ld_x, const T* w, int64_t ld_w, int32_t rows,
                                                    int64_t n, int64_t k, Epi epi) {
  constexpr int EPC = 16 / sizeof(T), kSlice = 4 * EPC, kWaves = 8, U = 4;
  __shared__ f32x4 sums[kWaves][TI * NI][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r = lane & 15;
  const int64_t j0 = (int64_t)blockIdx.x * (16 * NI);
  // Groups of U slices go to the waves in turn, so that a row's part that is
  // being read is one long run of memory.
  f32x4 acc[TI][NI] = {};
  // Whole aligned chunks come through buffer resources, where one that is
  // outside has its offset outside and is zero: no branch between the loads.
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<T*>(w + j0 * ld_w), (short)0, (int)0x80000000u, kBufferFlags);
  const __amdgpu_buffer_rsrc_t rx =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(x), (short)0, (int)0x80000000u, kBufferFlags);
  auto chunk = [&](const __amdgpu_buffer_rsrc_t& rsrc, const T* base, int64_t ld, int row, bool there, int64_t at) {
    u32x4 v = {0, 0, 0, 0};
    if constexpr (DIRECT) {
      const uint32_t off = (uint32_t)(row * (int)ld + (int)at) * (uint32_t)sizeof(T);
      v = __builtin_amdgcn_raw_buffer_load_b128(rsrc, there && at < k ? (int)off : (int)0x80000000u, 0, 0);
    } else {
      const int64_t left = there ? k - at : 0;
      const T* p = base + row * ld + at;
      if (left >= EPC) {
        __builtin_memcpy(&v, p, 16);
      } else if (left > 0) {
        T e[EPC];
#pragma unroll
        for (int t = 0; t < EPC; ++t) e[t] = t < left ? p[t] : (T)0;
        __builtin_memcpy(&v, e, 16);
      }
    }
    return v;
  };
  // The next group is on its way while one is multiplied.
  u32x4 fw[2][U][NI], fx[2][U][TI];
  auto load = [&](int to, int64_t at) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int b = 0; b < NI; ++b)
        fw[to][u][b] = chunk(rw, w + j0 * ld_w, ld_w, b * 16 + r, j0 + b * 16 + r < n, at + u * kSlice);
#pragma unroll
      for (int a = 0; a < TI; ++a) fx[to][u][a] = chunk(rx, x, ld_x, a * 16 + r, a * 16 + r < rows, at + u * kSlice);
    }
  };
  auto multiply = [&](int from) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int a = 0; a < TI; ++a)
#pragma unroll
        for (int b = 0; b < NI; ++b) acc[a][b] = mma_slice(fw[from][u][b], fx[from][u][a], acc[a][b], T{});
  };
  constexpr int64_t kGroup = kSlice * U, kTurn = kGroup * kWaves;
  const int64_t k0 = wave * kGroup;
  if (k0 < k) load(0, k0 + q * EPC);
  for (int64_t at = k0; at < k; at += 2 * kTurn) {
    load(1, at + kTurn + q * EPC);  // past the end: zeros, nothing read
    multiply(0);
    load(0, at + 2 * kTurn + q * EPC);
    multiply(1);
  }
#pragma unroll
  for (int a = 0; a < TI; ++a)
#pragma unroll
    for (int b = 0; b < NI; ++b) sums[wave][a * NI + b][lane] = acc[a][b];
  __syncthreads();
  // wave f adds up the blocks f, f + 8, ..
  for (int f = wave; f < TI * NI; f += kWaves) {
    f32x4 v = sums[0][f][lane];
#pragma unroll
    for (int s = 1; s < kWaves; ++s) v += sums[s][f][lane];
    const int64_t i = (f / NI) * 16 + r, j = j0 + (f % NI) * 16 + q * 4;
    if (i < rows && j < n) epi(i, j, v);
  }
}

constexpr int64_t kFewRows = 64;

// (A grid holds 2^32 threads; 2^26 outputs take 2^31.)
bool is_few(int64_t rows, int64_t n) { return rows <= kFewRows && n <= ((int64_t)1 << 26); }

template <class T, bool DIRECT, class Epi>
hipError_t few_rows(const void* x, int64_t ld_x, const void* w, int64_t ld_w, int64_t rows, int64_t n, int64_t k,
                    const Epi& epi, hipStream_t stream) {
  auto launch = [&](auto kernel, int per) {
    kernel<<<dim3((uint32_t)((n + per - 1) / per)), 512, 0, stream>>>(
        static_cast<const T*>(x), ld_x, static_cast<const T*>(w), ld_w, (int32_t)rows, n, k, epi);
  };
  if (rows <= 16) launch(k_linear_few<T, 1, 1, DIRECT, Epi>, 16);
  else if (rows <= 32) launch(k_linear_few<T, 2, 1, DIRECT, Epi>, 16);
  else launch(k_linear_few<T, 4, 2, DIRECT, Epi>, 32);
  return hipGetLastError();
}

// A 16-byte access at any address of an element.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// dz = dy act'(pre) and the column sums of dz, in strips of `strip` rows: one
// workgroup per 64 chunks of 16 bytes of columns and strip, a wave to a row
// and two rows in flight per wave.  dy and pre are read past the caches, dz
// is left in them for the products that read it next (8192 x 11008 bf16 when it
// was chosen, before the activations' ranges were widened: 103 us so, 155 us with
// ordinary loads, 109 us with the stores past them too).  Bound by those bytes:
// 541 MB in 110 to 115 us, 4.7 to 4.9 TB/s, with silu.  The
// strips' sums go to partial[strip][n] and are added in order by
// k_column_join, or straight to db when there is one strip.
template <class T, class G, int ACT>
__global__ void __launch_bounds__(256) k_bias_act(int64_t rows, int64_t n, const T* dy, int64_t ld_dy, const T* pre,
                                                  int64_t ld_pre, T* dz, int64_t ld_dz, float* partial,
                                                  G* db, int accumulate, int64_t strip) {
  constexpr int V = 16 / sizeof(T);
  __shared__ float sum[4][64][V + 1];
  const int c = threadIdx.x & 63, l = threadIdx.x >> 6;
  const int64_t j = ((int64_t)blockIdx.x * 64 + c) * V;
  const int64_t i0 = (int64_t)blockIdx.y * strip, i1 = i0 + strip < rows ? i0 + strip : rows;
  const int64_t left = n - j;
  float s[V] = {};
  if (left > 0) {
    auto load = [&](const T* p, T* to) {
      if (left >= V) {
        const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
        __builtin_memcpy(to, &v, 16);
      } else {
#pragma unroll
        for (int t = 0; t < V; ++t) to[t] = t < left ? p[t] : (T)0;
      }
    };
    // U rows' loads in flight at once
    constexpr int U = 2;
    for (int64_t i = i0 + l; i < i1; i += 4 * U) {
      T d[U][V], z[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + 4 * u < i1) {
          load(dy + (i + 4 * u) * ld_dy + j, d[u]);
          if constexpr (ACT != DC_ACT_NONE) load(pre + (i + 4 * u) * ld_pre + j, z[u]);
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + 4 * u < i1) {
          T o[V];
#pragma unroll
          for (int t = 0; t < V; ++t) {
            float v = (float)d[u][t];
            if constexpr (ACT != DC_ACT_NONE) v *= activation_slope((float)z[u][t], ACT);
            s[t] += v;
            o[t] = (T)v;
          }
          if (dz) {
            T* p = dz + (i + 4 * u) * ld_dz + j;
            if (left >= V) {
              __builtin_memcpy(p, o, 16);
            } else {
#pragma unroll
              for (int t = 0; t < V; ++t)
                if (t < left) p[t] = o[t];
            }
          }
        }
    }
  }
  if (!db) return;
#pragma unroll
  for (int t = 0; t < V; ++t) sum[l][c][t] = s[t];
  __syncthreads();
  for (int at = threadIdx.x; at < 64 * V; at += 256) {
    const int cc = at / V, t = at % V;
    const int64_t jj = ((int64_t)blockIdx.x * 64 + cc) * V + t;
    if (jj < n) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) v += sum[w][cc][t];
      if (gridDim.y > 1) partial[(int64_t)blockIdx.y * n + jj] = v;
      else db[jj] = (G)(accumulate ? (float)db[jj] + v : v);
    }
  }
}

// db from the strips' sums, eight lanes to a column, in a fixed order.  A few
// hundred KB: bound by latency, 3 to 5 us.
template <class G>
__global__ void __launch_bounds__(256) k_column_join(const float* partial, int32_t strips, int64_t n, G* db,
                                                     int accumulate) {
  __shared__ float sum[8][32];
  const int c = threadIdx.x & 31, l = threadIdx.x >> 5;
  const int64_t j = (int64_t)blockIdx.x * 32 + c;
  float v = 0.f;
  if (j < n)
    for (int32_t s = l; s < strips; s += 8) v += partial[(int64_t)s * n + j];
  sum[l][c] = v;
  __syncthreads();
  if (l == 0 && j < n) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += sum[w][c];
    db[j] = (G)(accumulate ? (float)db[j] + t : t);
  }
}

// Rows per strip: about 2048 workgroups over the chip, at least 32 rows each.
int64_t strip_rows(int32_t dtype, int64_t rows, int64_t n) {
  const int64_t per = dtype == DC_F32 ? 256 : 512;
  const int64_t across = (n + per - 1) / per;
  const int64_t strips = std::max<int64_t>(1, 2048 / across);
  const int64_t r = std::max<int64_t>(32, (rows + strips - 1) / strips);
  return (r + 7) / 8 * 8;
}

template <class T, class G>
hipError_t bias_act(int32_t dtype, int64_t rows, int64_t n, const void* dy, int64_t ld_dy, const void* pre,
                    int64_t ld_pre, int act, void* dz, int64_t ld_dz, void* db, int accumulate, float* partial,
                    hipStream_t stream) {
  const int64_t strip = strip_rows(dtype, rows, n);
  const int64_t strips = std::max<int64_t>(1, (rows + strip - 1) / strip);
  constexpr int64_t per = 64 * (16 / sizeof(T));
  const dim3 grid((uint32_t)((n + per - 1) / per), (uint32_t)strips);
  auto launch = [&](auto kernel) {
    kernel<<<grid, 256, 0, stream>>>(rows, n, static_cast<const T*>(dy), ld_dy, static_cast<const T*>(pre), ld_pre,
                                     static_cast<T*>(dz), ld_dz, partial, static_cast<G*>(db), accumulate, strip);
  };
  if (act == DC_ACT_RELU) launch(k_bias_act<T, G, DC_ACT_RELU>);
  else if (act == DC_ACT_GELU) launch(k_bias_act<T, G, DC_ACT_GELU>);
  else if (act == DC_ACT_SILU) launch(k_bias_act<T, G, DC_ACT_SILU>);
  else launch(k_bias_act<T, G, DC_ACT_NONE>);
  if (db && strips > 1)
    k_column_join<G><<<dim3((uint32_t)((n + 31) / 32)), 256, 0, stream>>>(partial, (int32_t)strips, n,
                                                                         static_cast<G*>(db), accumulate);
  return hipGetLastError();
}

}  // namespace

int64_t linear_workspace(int32_t dtype, int64_t T, int64_t N, int64_t K) {
  if (is_few(T, N)) return 0;
  return cut(dtype, T, N, K).partial_bytes(T);
}

int64_t linear_backward_workspace(int32_t dtype, int64_t T, int64_t N, int64_t K) {
  return std::max(cut(dtype, T, K, N).partial_bytes(T), cut(dtype, N, K, T).partial_bytes(N));
}

LaunchForm linear_form(int32_t dtype, int32_t kind, int64_t T, int64_t N, int64_t K) {
  if (kind == 0 && is_few(T, N)) return {};
  const int64_t m = kind == 2 ? N : T, n = kind == 0 ? N : K;
  const Cut c = cut(dtype, m, n, kind == 0 ? K : kind == 1 ? N : T);
  const int64_t tiles = ((m + c.tile - 1) / c.tile) * ((n + c.tile - 1) / c.tile);
  return {c.tile, launch_stages(c.tile, tiles * c.splits), c.splits};
}

int64_t bias_act_workspace(int32_t dtype, int64_t T, int64_t N) {
  const int64_t strip = strip_rows(dtype, T, N), strips = (T + strip - 1) / strip;
  return strips > 1 ? strips * N * 4 : 0;
}

hipError_t launch_linear(int32_t dtype, int64_t T, int64_t N, int64_t K, const void* x, int64_t ld_x, const void* w,
                         int64_t ld_w, const LinearOut& o, void* workspace, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  if (is_few(T, N)) {
    auto few = [&](auto type) {
      using E = decltype(type);
      const LinearEpilogue<E> epi{o, N};
      return direct_operand<E>(x, ld_x, K) && direct_operand<E>(w, ld_w, K)
                 ? few_rows<E, true>(x, ld_x, w, ld_w, T, N, K, epi, stream)
                 : few_rows<E, false>(x, ld_x, w, ld_w, T, N, K, epi, stream);
    };
    return dtype == DC_BF16 ? few(__bf16{}) : few(float{});
  }
  float* ws = static_cast<float*>(workspace);
  if (dtype == DC_BF16)
    return product<__bf16, true, true>(dtype, x, ld_x, w, ld_w, T, N, K, ws, LinearEpilogue<__bf16>{o, N}, stream);
  return product<float, true, true>(dtype, x, ld_x, w, ld_w, T, N, K, ws, LinearEpilogue<float>{o, N}, stream);
}

hipError_t launch_linear_dx(int32_t dtype, int64_t T, int64_t N, int64_t K, const void* dz, int64_t ld_dz,
                            const void* w, int64_t ld_w, const LinearOut& o, void* workspace, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  float* ws = static_cast<float*>(workspace);
  if (dtype == DC_BF16)
    return product<__bf16, true, false>(dtype, dz, ld_dz, w, ld_w, T, K, N, ws, GradEpilogue<__bf16>{o, K}, stream);
  return product<float, true, false>(dtype, dz, ld_dz, w, ld_w, T, K, N, ws, GradEpilogue<float>{o, K}, stream);
}

hipError_t launch_linear_dw(int32_t dtype, int32_t grad_dtype, int64_t T, int64_t N, int64_t K, const void* dz,
                            int64_t ld_dz, const void* x, int64_t ld_x, const LinearOut& o, void* workspace,
                            hipStream_t stream) {
  if (T == 0 && o.accumulate) return hipSuccess;
  float* ws = static_cast<float*>(workspace);
  if (dtype == DC_F32)
    return product<float, false, false>(dtype, dz, ld_dz, x, ld_x, N, K, T, ws, GradEpilogue<float>{o, K}, stream);
  if (grad_dtype == DC_F32)
    return product<__bf16, false, false>(dtype, dz, ld_dz, x, ld_x, N, K, T, ws, GradEpilogue<float>{o, K}, stream);
  return product<__bf16, false, false>(dtype, dz, ld_dz, x, ld_x, N, K, T, ws, GradEpilogue<__bf16>{o, K}, stream);
}

hipError_t launch_bias_act(int32_t dtype, int32_t grad_dtype, int64_t T, int64_t N, const void* dy, int64_t ld_dy,
                           const void* pre, int64_t ld_pre, int act, void* dz, int64_t ld_dz, void* db,
                           int accumulate, void* workspace, hipStream_t stream) {
  float* ws = static_cast<float*>(workspace);
  if (dtype == DC_F32)
    return bias_act<float, float>(dtype, T, N, dy, ld_dy, pre, ld_pre, act, dz, ld_dz, db, accumulate, ws, stream);
  if (grad_dtype == DC_F32)
    return bias_act<__bf16, float>(dtype, T, N, dy, ld_dy, pre, ld_pre, act, dz, ld_dz, db, accumulate, ws, stream);
  return bias_act<__bf16, __bf16>(dtype, T, N, dy, ld_dy, pre, ld_pre, act, dz, ld_dz, db, accumulate, ws, stream);
}

}  // namespace dc
