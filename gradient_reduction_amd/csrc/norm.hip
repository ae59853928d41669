// The root-mean-square norms after a block and before the next one, with the
// block's gate and the residual's scale, in one pass over a token's row:
//   u = (offset + post) h r1,   r1 = 1 / sqrt(mean(h^2) + eps)      (u = h without `post`)
//   s = x + scale gate u                                             (s = x without h)
//   y = (offset + gain) s r2,   r2 = 1 / sqrt(mean(s^2) + eps)
// and its backward, from dy and ds (the gradient that reaches s from later):
//   n = s r2,  q = (offset + gain) dy:   d = ds + r2 (q - n mean(q n)),  dgain (+)= sum_t dy n
//   dx = d,  du = scale gate d,  dgate (+)= sum_t scale d u
//   m = h r1,  g = (offset + post) du:   dh = r1 (g - m mean(g m)),      dpost (+)= sum_t du m
//
// A row is held in the registers of G threads, so every input is read once:
// forward 16 values each, backward 32 bytes of each operand (64 of fp32 rows of
// more than 8192).  Sums over a row are fp64, so that squares of any fp32 value
// neither overflow nor vanish.
//
// 8192 rows of 4096 bf16: forward 39 us (268 MB, 6.9 TB/s, bound by HBM);
// backward 74 to 79 and 5 for the join (403 MB, 5.1 to 5.4 TB/s), where the
// arithmetic of some 1000 instructions a wave and row (190 in fp64 and 83
// conversions to it) takes as long as the bytes and two waves a SIMD do not
// hide all of it.
// Tried: 8 values a thread instead of 16, twice the waves to a row, 111 to 119;
// one sum over the lanes in place of two (three more fp64 products a value in
// place of a second exchange), 95.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>
#include <utility>

#include "columns.h"
#include "device_common.h"
#include "internal.h"

namespace dc {
namespace {

constexpr int kEach = 16;  // values of a row per thread

// v and its partner's value added, for partners inside 16 lanes (CTRL: which),
// 16 or 32 lanes apart: register moves, where a shuffle goes through LDS.
template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
  const int2 x = __builtin_bit_cast(int2, v);
  const int2 y = {__builtin_amdgcn_update_dpp(0, x.x, CTRL, 0xf, 0xf, true),
                  __builtin_amdgcn_update_dpp(0, x.y, CTRL, 0xf, 0xf, true)};
  return v + __builtin_bit_cast(double, y);
}
template <int APART>
__device__ __forceinline__ double add_apart(double v) {
  const uint2 x = __builtin_bit_cast(uint2, v);
  uint2 a, b;
  if constexpr (APART == 16) {
    const auto lo = __builtin_amdgcn_permlane16_swap(x.x, x.x, false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(x.y, x.y, false, false);
    a = {lo[0], hi[0]}, b = {lo[1], hi[1]};
  } else {
    const auto lo = __builtin_amdgcn_permlane32_swap(x.x, x.x, false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap(x.y, x.y, false, false);
    a = {lo[0], hi[0]}, b = {lo[1], hi[1]};
  }
  return __builtin_bit_cast(double, a) + __builtin_bit_cast(double, b);
}
template <int G>
__device__ __forceinline__ double lanes_total(double v) {
  v = add_dpp<0xB1>(v);   // lane ^ 1
  v = add_dpp<0x4E>(v);   // lane ^ 2
  v = add_dpp<0x141>(v);  // mirrored in 8
  v = add_dpp<0x140>(v);  // mirrored in 16
  if constexpr (G >= 64) v = add_apart<32>(add_apart<16>(v));
  return v;
}

// Sums over the G threads of a row, N at once, to all of them.  With rows of
// more than a wave every thread of the workgroup must come, and `buf` is
// written anew: the caller keeps two calls on one buffer a barrier apart.
template <int G, int N, int THREADS>
__device__ __forceinline__ void row_total(double (&v)[N], double (*buf)[THREADS / 64]) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = lanes_total<G>(v[k]);
  if constexpr (G > 64) {
    constexpr int W = G / 64;
    const int wave = threadIdx.x >> 6, first = wave / W * W;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) buf[k][wave] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      double s = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) s += buf[k][first + w];
      v[k] = s;
    }
  }
}

// A row as a buffer: what lies past its columns, or of a row or an operand that
// is not there, loads as zeros and is not stored, without a branch.  (Behind a
// branch around a load every later wait is for all loads in flight, the next
// row's among them.)  For rows of whole 16 bytes; `row` is the wave's.
// The stores are streamed (nt): 8192 rows of 4096 bf16 backward take 84 us with
// it, 95 without, 89 with the loads streamed too.
constexpr int kStoreStream = 2;
template <class T>
struct RowBuffer {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ RowBuffer(const T* p, int64_t row, int64_t ld, int D, bool there) {
    r = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(p + (there ? row : 0) * ld), (short)0,
                                          p && there ? D * (int)sizeof(T) : 0, kBufferFlags);
  }
  __device__ __forceinline__ u32x4 load(int j) const {
    return __builtin_amdgcn_raw_buffer_load_b128(r, j * (int)sizeof(T), 0, 0);
  }
  template <int V>
  __device__ __forceinline__ void store(int j, const float (&v)[V]) const {
    T x[V];
#pragma unroll
    for (int t = 0; t < V; ++t) x[t] = (T)v[t];
    u32x4 w;
    __builtin_memcpy(&w, x, 16);
    __builtin_amdgcn_raw_buffer_store_b128(w, r, j * (int)sizeof(T), 0, kStoreStream);
  }
};

// One row of an operand, either way.
template <class T, int N, bool DIRECT>
__device__ __forceinline__ void load_row(Pack<T> (&v)[N], const T* p, int64_t row, int64_t ld, int D, bool there,
                                         int lane, int G) {
  if constexpr (DIRECT) {
    const RowBuffer<T> b(p, row, ld, D, there);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k].w = b.load((lane + G * k) * Pack<T>::V);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int j = (lane + G * k) * Pack<T>::V;
      v[k].w = u32x4{0, 0, 0, 0};
      if (p && there) v[k].load(p + row * ld + j, D - j);
    }
  }
}
template <class T, int N, int V, bool DIRECT>
__device__ __forceinline__ void store_row(const float (&v)[N][V], T* p, int64_t row, int64_t ld, int D, bool there,
                                          int lane, int G) {
  if constexpr (DIRECT) {
    const RowBuffer<T> b(p, row, ld, D, there);
#pragma unroll
    for (int k = 0; k < N; ++k) b.store((lane + G * k) * V, v[k]);
  } else {
    if (!p || !there) return;
#pragma unroll
    for (int k = 0; k < N; ++k) store_columns<T, V>(p + row * ld + (lane + G * k) * V, D - (lane + G * k) * V, v[k]);
  }
}

// 1 / sqrt(m) as r lift: the hardware's root where fp32 holds m well inside its
// range.  Of rows of subnormal values (with eps = 0) it passes fp32's range,
// though a value times it does not: r is then kLift times smaller.
constexpr float kLift = 4294967296.f;  // 2^32: the least rms, 2^-149 / sqrt(16384), gives r = 2^124
struct Root {
  float r, lift;
};
__device__ __forceinline__ Root inverse_root(double m) {
  if (m > 1e-30 && m < 1e30) return {__builtin_amdgcn_rsqf((float)m), 1.f};
  if (m < 1e-75) return {(float)(1.0 / (sqrt(m) * (double)kLift)), kLift};
  return {(float)(1.0 / sqrt(m)), 1.f};
}

template <class T>
struct NormIn {
  int64_t T_, D;
  const T *x, *h, *post, *gate, *gain;
  int64_t ld_x, ld_h, ld_gate, per_gate, gate_rows;  // per_gate: tokens per row of the gate
  float scale, offset;
  double eps, over;                       // over = 1 / D
  T *s, *y;
  int64_t ld_s, ld_y;
};

template <class T, int G, int THREADS, bool DIRECT>
__global__ void __launch_bounds__(THREADS) k_norm(NormIn<T> a) {
  constexpr int V = 16 / sizeof(T), N = kEach / V, ROWS = THREADS / G;
  __shared__ double buf[2][1][THREADS / 64];
  const int lane = threadIdx.x % G, D = (int)a.D;
  const int group = G < 64 ? threadIdx.x / G : __builtin_amdgcn_readfirstlane(threadIdx.x / G);
  for (int64_t row0 = (int64_t)blockIdx.x * ROWS; row0 < a.T_; row0 += (int64_t)gridDim.x * ROWS) {
    const int64_t row = row0 + group;
    const bool in = row < a.T_;
    Pack<T> x[N], h[N], post[N], gate[N], gain[N];
    load_row<T, N, DIRECT>(x, a.x, row, a.ld_x, D, in, lane, G);
    load_row<T, N, DIRECT>(h, a.h, row, a.ld_h, D, in, lane, G);
    load_row<T, N, DIRECT>(post, a.post, 0, 0, D, true, lane, G);
    load_row<T, N, DIRECT>(gate, a.gate, in && a.gate_rows > 1 ? row / a.per_gate : 0, a.ld_gate, D, true, lane, G);
    load_row<T, N, DIRECT>(gain, a.gain, 0, 0, D, true, lane, G);
    float s[N][V];
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int t = 0; t < V; ++t) s[k][t] = x[k][t];
    if (a.h) {
      Root root = {1.f, 1.f};
      if (a.post) {
        double sum[1] = {0};
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
          for (int t = 0; t < V; ++t) {
            const double v = h[k][t];
            sum[0] = __builtin_fma(v, v, sum[0]);
          }
        row_total<G, 1, THREADS>(sum, buf[0]);
        root = inverse_root(__builtin_fma(sum[0], a.over, a.eps));
      }
      const float scale = a.scale * root.lift;
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int t = 0; t < V; ++t) {
          float u = h[k][t] * root.r;
          if (a.post) u *= a.offset + post[k][t];
          u *= scale;
          if (a.gate) u *= gate[k][t];
          s[k][t] += u;
        }
      store_row<T, N, V, DIRECT>(s, a.s, row, a.ld_s, D, in, lane, G);
    }
    if (a.gain) {
      double sum[1] = {0};
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int t = 0; t < V; ++t) sum[0] = __builtin_fma((double)s[k][t], (double)s[k][t], sum[0]);
      row_total<G, 1, THREADS>(sum, buf[1]);
      const Root root = inverse_root(__builtin_fma(sum[0], a.over, a.eps));
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int t = 0; t < V; ++t) s[k][t] = s[k][t] * root.r * root.lift * (a.offset + gain[k][t]);
      store_row<T, N, V, DIRECT>(s, a.y, row, a.ld_y, D, in, lane, G);
    }
    if constexpr (G > 64) __syncthreads();  // buf is free for the next row
  }
}

template <class T, class G_>
struct NormBack {
  int64_t T_, D;
  const T *dy, *ds, *s, *h, *post, *gate, *gain;
  int64_t ld_dy, ld_ds, ld_s, ld_h, ld_gate, per_gate;
  float scale, offset;
  double eps, over;
  T *dx, *dh;
  int64_t ld_dx, ld_dh;
  G_* dgate;             // written here where several rows of the gate end inside a run
  int64_t ld_dgate;
  int32_t accumulate, sums_post, sums_gate;
  int64_t run;           // rows per run
  float* partial;        // [2][workgroups][D]: of dgain; of dpost, or of sum_t d m
  float* gate_partial;   // [runs][2][D]: of a gate row that came into the run, of one that goes on
};

// Adds every row group's column sums up in `cols` (LDS) and writes them.
template <class T, int G, int EACH, int THREADS>
__device__ __forceinline__ void columns_out(float (&sum)[EACH], float* cols, float* to, int64_t D) {
  constexpr int V = 16 / sizeof(T), ROWS = THREADS / G;
  const int lane = threadIdx.x % G, mine = threadIdx.x / G;
  auto at = [&](int e) { return (lane + G * (e / V)) * V + e % V; };
  if constexpr (ROWS == 1) {
#pragma unroll
    for (int e = 0; e < EACH; ++e)
      if (at(e) < D) to[at(e)] = sum[e];
  } else {
    for (int r = 0; r < ROWS; ++r) {
      if (mine == r)
#pragma unroll
        for (int e = 0; e < EACH; ++e) cols[at(e)] = r ? cols[at(e)] + sum[e] : sum[e];
      __syncthreads();
    }
    for (int64_t j = threadIdx.x; j < D; j += THREADS) to[j] = cols[j];
    __syncthreads();
  }
}

// What the backward reads of a token's row.
template <class T, int N>
struct BackRow {
  Pack<T> s[N], dy[N], ds[N], h[N];
};

// Every row group takes a run of neighbouring rows and keeps the column sums of
// the parameters' gradients in registers; the next row's loads are under way
// while a row is worked on (not in workgroups of 1024: their threads have 128
// registers, and spill without it already).  GATES: the
// gate has several rows; its sums are handed out where a gate row ends.
// Without, sum_t d m is kept, which gives dpost and dgate both (k_norm_join).
template <class T, class G_, int G, int EACH, int THREADS, bool GATES, bool DIRECT>
__global__ void __launch_bounds__(THREADS) k_norm_back(NormBack<T, G_> a) {
  constexpr int V = 16 / sizeof(T), N = EACH / V, ROWS = THREADS / G;
  constexpr bool AHEAD = THREADS <= 512;
  __shared__ double buf[2][3][THREADS / 64];
  __shared__ float cols[ROWS == 1 ? 1 : G * EACH];
  const int lane = threadIdx.x % G, D = (int)a.D;
  // (a wave is of one row: what follows from it is scalar)
  const int group = G < 64 ? threadIdx.x / G : __builtin_amdgcn_readfirstlane(threadIdx.x / G);
  const int64_t run = (int64_t)blockIdx.x * ROWS + group, first = run * a.run;
  const int64_t end = first + a.run < a.T_ ? first + a.run : a.T_;
  float sum_gain[EACH] = {}, sum_post[EACH] = {}, sum_gate[GATES ? EACH : 1] = {};
  auto load = [&](BackRow<T, N>& r, int64_t row) {
    const bool in = row < end;
    load_row<T, N, DIRECT>(r.s, a.s, row, a.ld_s, D, in, lane, G);
    load_row<T, N, DIRECT>(r.dy, a.dy, row, a.ld_dy, D, in, lane, G);
    load_row<T, N, DIRECT>(r.h, a.h, row, a.ld_h, D, in, lane, G);
    load_row<T, N, DIRECT>(r.ds, a.ds, row, a.ld_ds, D, in, lane, G);
  };
  // The vectors as they multiply, in fp32 for the whole run: offset + gain, and
  // 1 where there is none.
  float gain[N][V], post[N][V], gate[N][V];
  auto vector = [&](float (&to)[N][V], const T* p, int64_t row, int64_t ld, float offset) {
    Pack<T> v[N];
    load_row<T, N, DIRECT>(v, p, row, ld, D, true, lane, G);
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int t = 0; t < V; ++t) to[k][t] = p ? offset + v[k][t] : 1.f;
  };
  vector(gain, a.gain, 0, 0, a.offset);
  vector(post, a.post, 0, 0, a.offset);
  if constexpr (!GATES) vector(gate, a.gate, 0, 0, 0.f);
  BackRow<T, N> cur;
  load(cur, first);
  for (int64_t i = 0; i < a.run; ++i) {
    const int64_t row = first + i;
    const bool in = row < end;
    BackRow<T, N> next;
    if constexpr (AHEAD) load(next, row + 1);
    float d[N][V];
    double sum[3] = {0, 0, 0};
    if (a.gain) {
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int t = 0; t < V; ++t) {
          const double v = cur.s[k][t], q = cur.dy[k][t] * gain[k][t];
          sum[0] = __builtin_fma(v, v, sum[0]);
          sum[1] = __builtin_fma(q, v, sum[1]);
        }
    }
    if (a.post) {
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int t = 0; t < V; ++t) {
          const double v = cur.h[k][t];
          sum[2] = __builtin_fma(v, v, sum[2]);
        }
    }
    row_total<G, 3, THREADS>(sum, buf[0]);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      cur.s[k].forget(), cur.dy[k].forget(), cur.h[k].forget();
#pragma unroll
      for (int t = 0; t < V; ++t) d[k][t] = cur.ds[k][t];
    }
    if (a.gain) {
      // (a row past the last one adds zeros, whatever eps is)
      // lifted: n is `lift` times too small, y and q that many times too large
      const Root root = in ? inverse_root(__builtin_fma(sum[0], a.over, a.eps)) : Root{0.f, 1.f};
      const float r = root.r, mean = (float)(sum[1] * a.over * r * (double)(root.lift * root.lift * root.lift));
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int t = 0; t < V; ++t) {
          const float n = cur.s[k][t] * r, y = cur.dy[k][t] * root.lift, q = y * gain[k][t];
          sum_gain[k * V + t] = __builtin_fmaf(y, n, sum_gain[k * V + t]);
          d[k][t] = __builtin_fmaf(r, q - n * mean, d[k][t]);
        }
    }
    store_row<T, N, V, DIRECT>(d, a.dx, row, a.ld_dx, D, in, lane, G);
    if (a.h) {
      // lifted: m is `lift` times too small, e, v, du and g that many times too large
      const Root root = !in ? Root{0.f, 1.f} : a.post ? inverse_root(__builtin_fma(sum[2], a.over, a.eps)) : Root{1.f, 1.f};
      const float r = root.r;
      const int64_t gate_row = GATES && in ? row / a.per_gate : 0;
      if constexpr (GATES) vector(gate, a.gate, gate_row, a.ld_gate, 0.f);
      float g[N][V];
      double dot[1] = {0};
#pragma unroll
      for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int t = 0; t < V; ++t) {
          const float m = cur.h[k][t] * r, w = post[k][t], e = root.lift * d[k][t], v = a.scale * e, du = v * gate[k][t];
          if constexpr (GATES) {
            sum_post[k * V + t] = __builtin_fmaf(du, m, sum_post[k * V + t]);
            sum_gate[k * V + t] = __builtin_fmaf(v, m * w, sum_gate[k * V + t]);
          } else {
            sum_post[k * V + t] = __builtin_fmaf(e, m, sum_post[k * V + t]);
          }
          g[k][t] = du * w;
          dot[0] = __builtin_fma((double)g[k][t], (double)m, dot[0]);
        }
      }
      if (a.post) {  // (without it g is dh, whatever stands in h)
        row_total<G, 1, THREADS>(dot, buf[1]);
        const float mean = (float)(dot[0] * a.over * (double)(root.lift * root.lift));
#pragma unroll
        for (int k = 0; k < N; ++k) cur.h[k].forget();
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
          for (int t = 0; t < V; ++t) g[k][t] = r * (g[k][t] - cur.h[k][t] * r * mean);
      }
      store_row<T, N, V, DIRECT>(g, a.dh, row, a.ld_dh, D, in, lane, G);
      if constexpr (GATES) {
        const int64_t g0 = gate_row * a.per_gate, g1 = g0 + a.per_gate;
        if (a.sums_gate && in && (row + 1 == g1 || row + 1 == end)) {
          const bool here = g0 >= first && g1 <= end;
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const int j = (lane + G * k) * V, left = D - j;
            float v[V];
#pragma unroll
            for (int t = 0; t < V; ++t) v[t] = sum_gate[k * V + t];
            if (here) {
              G_* to = a.dgate + gate_row * a.ld_dgate + j;
              if (a.accumulate) {
                float old[V];
                load_columns<G_, V>(to, left, old);
#pragma unroll
                for (int t = 0; t < V; ++t) v[t] += old[t];
              }
              store_columns<G_, V>(to, left, v);
            } else {
              store_columns<float, V>(a.gate_partial + (run * 2 + (g0 >= first ? 1 : 0)) * a.D + j, left, v);
            }
          }
#pragma unroll
          for (int e = 0; e < EACH; ++e) sum_gate[e] = 0.f;
        }
      }
    }
    if constexpr (G > 64) __syncthreads();
    if constexpr (AHEAD) cur = next;
    else load(cur, row + 1);
  }
  if (a.gain) columns_out<T, G, EACH, THREADS>(sum_gain, cols, a.partial + (int64_t)blockIdx.x * a.D, a.D);
  if (a.sums_post)
    columns_out<T, G, EACH, THREADS>(sum_post, cols, a.partial + ((int64_t)gridDim.x + blockIdx.x) * a.D, a.D);
}

template <class T, class G_>
struct NormJoin {
  int64_t D;
  const float* partial;
  int32_t blocks, gates;
  const T *post, *gate;
  float scale, offset;
  G_ *dgain, *dpost, *dgate;  // dgate: of a gate of one row
  int32_t accumulate, from;
};

// Column sums of the workgroups in order, eight lanes to a column.  blockIdx.y,
// from `from` on: 0 dgain, 1 dpost and a single gate row's gradient.
template <class T, class G_>
__global__ void __launch_bounds__(256) k_norm_join(NormJoin<T, G_> a) {
  __shared__ float sum[8][32];
  const int c = threadIdx.x & 31, l = threadIdx.x >> 5;
  const int64_t j = (int64_t)blockIdx.x * 32 + c;
  const int which = a.from + (int)blockIdx.y;
  const float* p = a.partial + (int64_t)which * a.blocks * a.D;
  float v = 0.f;
  if (j < a.D) {
#pragma unroll 16
    for (int32_t b = l; b < a.blocks; b += 8) v += p[b * a.D + j];
  }
  sum[l][c] = v;
  __syncthreads();
  if (l || j >= a.D) return;
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) t += sum[w][c];
  auto put = [&](G_* to, float v) { to[j] = (G_)(a.accumulate ? (float)to[j] + v : v); };
  if (which == 0) {
    put(a.dgain, t);
  } else if (a.gates) {
    put(a.dpost, t);
  } else {
    if (a.dpost) put(a.dpost, a.gate ? a.scale * t * (float)a.gate[j] : a.scale * t);
    if (a.dgate) put(a.dgate, a.post ? a.scale * t * (a.offset + (float)a.post[j]) : a.scale * t);
  }
}

// Gate rows that reach over runs: their parts in order, in fp64, so that
// thousands of them (narrow rows have runs of one or two) add no error that grows with
// their number.  (No tokens: zeros.)
template <class G_>
__global__ void __launch_bounds__(256) k_gate_join(int64_t D, int64_t T_, int64_t rows, int64_t run, int64_t per_gate,
                                                   const float* partial, G_* dgate, int64_t ld, int32_t accumulate) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= D) return;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const int64_t g0 = row * per_gate, r0 = g0 / run, r1 = (g0 + per_gate - 1) / run;
    if (T_ && r0 == r1) continue;
    double v = 0;
    if (T_) {
#pragma unroll 8
      for (int64_t r = r0; r <= r1; ++r) v += partial[(r * 2 + (r == r0 ? 1 : 0)) * D + j];
    }
    G_* to = dgate + row * ld + j;
    *to = (G_)(float)(accumulate ? (double)(float)*to + v : v);
  }
}

// Threads per row: the fewest of a few steps that hold it.  Forward a thread
// takes 16 values (with four times the threads 65536 rows of 256 bf16 took 53 us
// for 29, 32768 of 1024 93 for 45, 8192 of 4096 143 for 44; fp32 59 for 45, 110
// for 81, 167 for 80).  Between the steps lanes are left without columns: as
// many bytes in rows of 2048 take 63 us, of 5120 118, of 8192 80, of 4096 45.
// Backward a thread takes 32 bytes of a row of each operand (64 for fp32 rows of
// more than 8192), and a workgroup 512 threads: two waves a SIMD, whose 256
// registers hold two rows' operands and the sums (bf16 with the next step's
// threads: 65536 x 256 95 us for 53, 32768 x 1024 205 for 85, 8192 x 4096 119 for
// 80, 4096 x 8192 632 for 88).
int row_threads(int64_t D) { return D <= 256 ? 16 : D <= 1024 ? 64 : D <= 4096 ? 256 : 1024; }
int back_row_threads(int32_t dtype, int64_t D) {
  const int64_t n = dtype == DC_BF16 ? 16 : 8;
  return D <= 16 * n ? 16 : D <= 64 * n ? 64 : D <= 256 * n ? 256 : D <= 512 * n ? 512 : 1024;
}
constexpr int back_threads(int g) { return g > 512 ? g : 512; }

// Runs of the backward: about one workgroup a compute unit, each row group
// with as few rows as that leaves (half and twice as many workgroups: 8192 x
// 4096 bf16 119 and 86 us where 256 take 80, 65536 x 256 69 and 67 for 53, 4096 x
// 4096 fp32 97 and 80 for 77).
constexpr int64_t kBlocks = 256;
struct Runs {
  int64_t rows, count, blocks;
  Runs(int32_t dtype, int64_t T, int64_t D) {
    const int g = back_row_threads(dtype, D);
    const int64_t groups = back_threads(g) / g;
    rows = std::max<int64_t>(1, (T + kBlocks * groups - 1) / (kBlocks * groups));
    count = (T + rows - 1) / rows;
    blocks = std::max<int64_t>(1, (count + groups - 1) / groups);
  }
};

// Whether rows are whole 16 bytes apart and long, from a 16-byte boundary.
template <class T>
bool direct_rows(int64_t D, std::initializer_list<std::pair<const void*, int64_t>> rows) {
  bool yes = D % Pack<T>::V == 0;
  for (const auto& r : rows)
    yes &= r.first == nullptr || (reinterpret_cast<uintptr_t>(r.first) % 16 == 0 && r.second % Pack<T>::V == 0);
  return yes;
}

template <class T>
hipError_t norm(const NormLaunch& l, hipStream_t stream) {
  NormIn<T> a{};
  a.T_ = l.T;
  a.D = l.D;
  a.x = static_cast<const T*>(l.x);
  a.h = static_cast<const T*>(l.h);
  a.post = static_cast<const T*>(l.post);
  a.gate = static_cast<const T*>(l.gate);
  a.gain = static_cast<const T*>(l.gain);
  a.ld_x = l.ld_x;
  a.ld_h = l.ld_h;
  a.ld_gate = l.ld_gate;
  a.per_gate = std::max<int64_t>(1, l.T / l.gate_rows);
  a.scale = l.scale;
  a.offset = l.offset;
  a.eps = l.eps;
  a.over = 1.0 / (double)l.D;
  a.s = static_cast<T*>(l.out_s);
  a.y = static_cast<T*>(l.y);
  a.ld_s = l.ld_out_s;
  a.ld_y = l.ld_y;
  a.gate_rows = l.gate_rows;
  const bool direct = direct_rows<T>(l.D, {{l.x, l.ld_x}, {l.h, l.ld_h}, {l.post, 0}, {l.gain, 0},
                                           {l.gate, l.gate_rows > 1 ? l.ld_gate : 0}, {l.out_s, l.ld_out_s}, {l.y, l.ld_y}});
  auto launch = [&](auto g) {
    constexpr int kG = decltype(g)::value, kThreads = kG > 256 ? kG : 256, kRows = kThreads / kG;
    auto kernel = k_norm<T, kG, kThreads, false>;
    if constexpr (kG >= 64) {  // (a row to a wave)
      if (direct) kernel = k_norm<T, kG, kThreads, true>;
    }
    const int64_t blocks = std::min<int64_t>((l.T + kRows - 1) / kRows, (int64_t)1 << 20);
    kernel<<<dim3((uint32_t)blocks), kThreads, 0, stream>>>(a);
  };
  switch (row_threads(l.D)) {
    case 16: launch(std::integral_constant<int, 16>{}); break;
    case 64: launch(std::integral_constant<int, 64>{}); break;
    case 256: launch(std::integral_constant<int, 256>{}); break;
    default: launch(std::integral_constant<int, 1024>{}); break;
  }
  return hipGetLastError();
}

template <class T, class G_>
hipError_t norm_back(const NormLaunch& l, hipStream_t stream) {
  const Runs runs(l.dtype, l.T, l.D);
  const bool gates = l.gate && l.gate_rows > 1;
  NormBack<T, G_> a{};
  a.T_ = l.T;
  a.D = l.D;
  a.dy = static_cast<const T*>(l.gain ? l.dy : nullptr);
  a.ds = static_cast<const T*>(l.ds);
  a.s = static_cast<const T*>(l.gain ? l.x : nullptr);
  a.h = static_cast<const T*>(l.h);
  a.post = static_cast<const T*>(l.post);
  a.gate = static_cast<const T*>(l.gate);
  a.gain = static_cast<const T*>(l.gain);
  a.ld_dy = l.ld_dy;
  a.ld_ds = l.ld_ds;
  a.ld_s = l.ld_x;
  a.ld_h = l.ld_h;
  a.ld_gate = l.ld_gate;
  a.per_gate = std::max<int64_t>(1, l.T / l.gate_rows);
  a.scale = l.scale;
  a.offset = l.offset;
  a.eps = l.eps;
  a.over = 1.0 / (double)l.D;
  a.dx = static_cast<T*>(l.dx);
  a.dh = static_cast<T*>(l.dh);
  a.ld_dx = l.ld_dx;
  a.ld_dh = l.ld_dh;
  a.dgate = static_cast<G_*>(l.dgate);
  a.ld_dgate = l.ld_dgate;
  a.accumulate = l.accumulate;
  a.sums_post = l.dpost || (l.dgate && !gates);
  a.sums_gate = l.dgate != nullptr;
  a.run = runs.rows;
  a.partial = static_cast<float*>(l.workspace);
  a.gate_partial = a.partial + 2 * runs.blocks * l.D;
  const bool direct = direct_rows<T>(
      l.D, {{a.dy, l.ld_dy}, {l.ds, l.ld_ds}, {a.s, l.ld_x}, {l.h, l.ld_h}, {l.post, 0}, {l.gain, 0},
            {l.gate, gates ? l.ld_gate : 0}, {l.dx, l.ld_dx}, {l.dh, l.ld_dh}});
  auto launch = [&](auto g, auto each) {
    constexpr int kG = decltype(g)::value, kE = decltype(each)::value, kThreads = back_threads(kG);
    auto kernel = k_norm_back<T, G_, kG, kE, kThreads, false, false>;
    if (gates) kernel = k_norm_back<T, G_, kG, kE, kThreads, true, false>;
    if constexpr (kG >= 64) {  // (a row to a wave)
      if (direct && gates) kernel = k_norm_back<T, G_, kG, kE, kThreads, true, true>;
      else if (direct) kernel = k_norm_back<T, G_, kG, kE, kThreads, false, true>;
    }
    kernel<<<dim3((uint32_t)runs.blocks), kThreads, 0, stream>>>(a);
  };
  constexpr std::integral_constant<int, 32 / sizeof(T)> each;
  switch (back_row_threads(l.dtype, l.D)) {
    case 16: launch(std::integral_constant<int, 16>{}, each); break;
    case 64: launch(std::integral_constant<int, 64>{}, each); break;
    case 256: launch(std::integral_constant<int, 256>{}, each); break;
    case 512: launch(std::integral_constant<int, 512>{}, each); break;
    default:
      if (l.D <= 1024 * each) launch(std::integral_constant<int, 1024>{}, each);
      else launch(std::integral_constant<int, 1024>{}, std::integral_constant<int, kEach>{});
  }
  NormJoin<T, G_> j{};
  j.D = l.D;
  j.partial = a.partial;
  j.blocks = (int32_t)runs.blocks;
  j.gates = gates;
  j.post = a.post;
  j.gate = a.gate;
  j.scale = l.scale;
  j.offset = l.offset;
  j.dgain = static_cast<G_*>(l.dgain);
  j.dpost = static_cast<G_*>(l.dpost);
  j.dgate = a.dgate;
  j.accumulate = l.accumulate;
  j.from = l.dgain ? 0 : 1;
  const uint32_t sums = (l.dgain ? 1 : 0) + (a.sums_post ? 1 : 0);
  if (sums) k_norm_join<T, G_><<<dim3((uint32_t)((l.D + 31) / 32), sums), 256, 0, stream>>>(j);
  // a run of whole gate rows has written them all
  if (gates && l.dgate && (l.T == 0 || runs.rows % a.per_gate != 0))
    k_gate_join<G_><<<dim3((uint32_t)((l.D + 255) / 256), (uint32_t)std::min<int64_t>(l.gate_rows, 32768)), 256, 0,
                      stream>>>(l.D, l.T, l.gate_rows, runs.rows, a.per_gate, a.gate_partial, a.dgate, l.ld_dgate,
                                l.accumulate);
  return hipGetLastError();
}

}  // namespace

int64_t norm_most_columns() { return 1024 * kEach; }

int64_t norm_workspace(int32_t dtype, int64_t T, int64_t D, int64_t gate_rows) {
  const Runs runs(dtype, T, D);
  return 4 * D * (2 * runs.blocks + (gate_rows > 1 ? 2 * runs.count : 0));
}

hipError_t launch_norm(const NormLaunch& l, hipStream_t stream) {
  if (l.T == 0) return hipSuccess;
  return l.dtype == DC_BF16 ? norm<__bf16>(l, stream) : norm<float>(l, stream);
}

hipError_t launch_norm_backward(const NormLaunch& l, hipStream_t stream) {
  if (l.dtype == DC_F32) return norm_back<float, float>(l, stream);
  if (l.grad_dtype == DC_F32) return norm_back<__bf16, float>(l, stream);
  return norm_back<__bf16, __bf16>(l, stream);
}

}  // namespace dc
