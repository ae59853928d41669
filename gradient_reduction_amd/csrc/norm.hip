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
// A row is held in the registers of G threads, 16 values each, so every input
// is read once.  Sums over a row are fp64, so that squares of any fp32 value
// neither overflow nor vanish.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "columns.h"
#include "device_common.h"
#include "internal.h"

namespace dc {
namespace {

constexpr int kEach = 16;  // values of a row per thread

// Sums over the G threads of a row, N at once, to all of them.  With rows of
// more than a wave every thread of the workgroup must come, and `buf` is
// written anew: the caller keeps two calls on one buffer a barrier apart.
template <int G, int N, int THREADS>
__device__ __forceinline__ void row_total(double (&v)[N], double (*buf)[THREADS / 64]) {
#pragma unroll
  for (int o = (G < 64 ? G : 64) / 2; o; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], o);
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

// 1 / sqrt(m): the hardware's where fp32 holds m well inside its range.
__device__ __forceinline__ float inverse_root(double m) {
  if (m > 1e-30 && m < 1e30) return __builtin_amdgcn_rsqf((float)m);
  return (float)(1.0 / sqrt(m));
}

template <class T>
struct NormIn {
  int64_t T_, D;
  const T *x, *h, *post, *gate, *gain;
  int64_t ld_x, ld_h, ld_gate, per_gate;  // tokens per row of the gate
  float scale, offset;
  double eps, over;                       // over = 1 / D
  T *s, *y;
  int64_t ld_s, ld_y;
};

template <class T, int G, int THREADS>
__global__ void __launch_bounds__(THREADS) k_norm(NormIn<T> a) {
  constexpr int V = 16 / sizeof(T), N = kEach / V, ROWS = THREADS / G;
  __shared__ double buf[2][1][THREADS / 64];
  const int lane = threadIdx.x % G;
  for (int64_t row0 = (int64_t)blockIdx.x * ROWS; row0 < a.T_; row0 += (int64_t)gridDim.x * ROWS) {
    const int64_t row = row0 + threadIdx.x / G;
    const bool in = row < a.T_;
    float s[N][V];
    {
      Pack<T> x[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int64_t j = (int64_t)(lane + G * k) * V;
        x[k].load(a.x + row * a.ld_x + j, in ? a.D - j : 0);
#pragma unroll
        for (int t = 0; t < V; ++t) s[k][t] = x[k][t];
      }
    }
    if (a.h) {
      Pack<T> h[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int64_t j = (int64_t)(lane + G * k) * V;
        h[k].load(a.h + row * a.ld_h + j, in ? a.D - j : 0);
      }
      float r = 1.f;
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
        r = inverse_root(__builtin_fma(sum[0], a.over, a.eps));
      }
      const T* gate = a.gate ? a.gate + (in ? row / a.per_gate : 0) * a.ld_gate : nullptr;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int64_t j = (int64_t)(lane + G * k) * V, left = in ? a.D - j : 0;
        Pack<T> p, g;
        if (a.post) p.load(a.post + j, left);
        if (gate) g.load(gate + j, left);
#pragma unroll
        for (int t = 0; t < V; ++t) {
          float u = h[k][t] * r;
          if (a.post) u *= a.offset + p[t];
          u *= a.scale;
          if (gate) u *= g[t];
          s[k][t] += u;
        }
        if (a.s) store_columns<T, V>(a.s + row * a.ld_s + j, left, s[k]);
      }
    }
    if (a.gain) {
      double sum[1] = {0};
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int t = 0; t < V; ++t) sum[0] = __builtin_fma((double)s[k][t], (double)s[k][t], sum[0]);
      row_total<G, 1, THREADS>(sum, buf[1]);
      const float r = inverse_root(__builtin_fma(sum[0], a.over, a.eps));
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int64_t j = (int64_t)(lane + G * k) * V, left = in ? a.D - j : 0;
        Pack<T> p;
        p.load(a.gain + j, left);
#pragma unroll
        for (int t = 0; t < V; ++t) s[k][t] = s[k][t] * r * (a.offset + p[t]);
        store_columns<T, V>(a.y + row * a.ld_y + j, left, s[k]);
      }
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
template <class T, int G, int THREADS>
__device__ __forceinline__ void columns_out(float (&sum)[kEach], float* cols, float* to, int64_t D) {
  constexpr int V = 16 / sizeof(T), ROWS = THREADS / G;
  const int lane = threadIdx.x % G, mine = threadIdx.x / G;
  auto at = [&](int e) { return (lane + G * (e / V)) * V + e % V; };
  if constexpr (ROWS == 1) {
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (at(e) < D) to[at(e)] = sum[e];
  } else {
    for (int r = 0; r < ROWS; ++r) {
      if (mine == r)
#pragma unroll
        for (int e = 0; e < kEach; ++e) cols[at(e)] = r ? cols[at(e)] + sum[e] : sum[e];
      __syncthreads();
    }
    for (int64_t j = threadIdx.x; j < D; j += THREADS) to[j] = cols[j];
    __syncthreads();
  }
}

// Every row group takes a run of neighbouring rows and keeps the column sums of
// the parameters' gradients in registers.  GATES: the gate has several rows;
// its sums are handed out where a gate row ends.  Without, sum_t d m is kept,
// which gives dpost and dgate both (k_norm_join).
template <class T, class G_, int G, int THREADS, bool GATES>
__global__ void __launch_bounds__(THREADS) k_norm_back(NormBack<T, G_> a) {
  constexpr int V = 16 / sizeof(T), N = kEach / V, ROWS = THREADS / G;
  __shared__ double buf[2][3][THREADS / 64];
  __shared__ float cols[ROWS == 1 ? 1 : G * kEach];
  const int lane = threadIdx.x % G;
  const int64_t run = (int64_t)blockIdx.x * ROWS + threadIdx.x / G, first = run * a.run;
  const int64_t end = first + a.run < a.T_ ? first + a.run : a.T_;
  float sum_gain[kEach] = {}, sum_post[kEach] = {}, sum_gate[GATES ? kEach : 1] = {};
  for (int64_t i = 0; i < a.run; ++i) {
    const int64_t row = first + i;
    const bool in = row < a.T_;
    Pack<T> s[N], dy[N], h[N];
    float d[N][V];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int64_t j = (int64_t)(lane + G * k) * V, left = in ? a.D - j : 0;
      if (a.gain) {
        s[k].load(a.s + row * a.ld_s + j, left);
        dy[k].load(a.dy + row * a.ld_dy + j, left);
      }
      if (a.h) h[k].load(a.h + row * a.ld_h + j, left);
      Pack<T> v;
      v.w = u32x4{0, 0, 0, 0};
      if (a.ds) v.load(a.ds + row * a.ld_ds + j, left);
#pragma unroll
      for (int t = 0; t < V; ++t) d[k][t] = v[t];
    }
    double sum[3] = {0, 0, 0};
    if (a.gain) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int64_t j = (int64_t)(lane + G * k) * V;
        Pack<T> p;
        p.load(a.gain + j, a.D - j);
#pragma unroll
        for (int t = 0; t < V; ++t) {
          const double v = s[k][t], q = dy[k][t] * (a.offset + p[t]);
          sum[0] = __builtin_fma(v, v, sum[0]);
          sum[1] = __builtin_fma(q, v, sum[1]);
        }
      }
    }
    if (a.post) {
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int t = 0; t < V; ++t) {
          const double v = h[k][t];
          sum[2] = __builtin_fma(v, v, sum[2]);
        }
    }
    row_total<G, 3, THREADS>(sum, buf[0]);
    if (a.gain) {
      // (a row past the last one adds zeros, whatever eps is)
      const float r = in ? inverse_root(__builtin_fma(sum[0], a.over, a.eps)) : 0.f;
      const float mean = (float)(sum[1] * a.over * r);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int64_t j = (int64_t)(lane + G * k) * V;
        Pack<T> p;
        p.load(a.gain + j, a.D - j);
#pragma unroll
        for (int t = 0; t < V; ++t) {
          const float n = s[k][t] * r, q = dy[k][t] * (a.offset + p[t]);
          sum_gain[k * V + t] += dy[k][t] * n;
          d[k][t] += r * (q - n * mean);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int64_t j = (int64_t)(lane + G * k) * V, left = in ? a.D - j : 0;
      if (a.dx) store_columns<T, V>(a.dx + row * a.ld_dx + j, left, d[k]);
    }
    if (a.h) {
      const float r = !in ? 0.f : a.post ? inverse_root(__builtin_fma(sum[2], a.over, a.eps)) : 1.f;
      const int64_t gate_row = GATES && in ? row / a.per_gate : 0;
      const T* gate = a.gate ? a.gate + gate_row * a.ld_gate : nullptr;
      float g[N][V];
      double dot[1] = {0};
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int64_t j = (int64_t)(lane + G * k) * V;
        Pack<T> p, w;
        if (a.post) p.load(a.post + j, a.D - j);
        if (gate) w.load(gate + j, a.D - j);
#pragma unroll
        for (int t = 0; t < V; ++t) {
          const float m = h[k][t] * r, gain = a.post ? a.offset + p[t] : 1.f;
          const float du = a.scale * d[k][t] * (gate ? w[t] : 1.f);
          if constexpr (GATES) {
            sum_post[k * V + t] += du * m;
            sum_gate[k * V + t] += a.scale * d[k][t] * (m * gain);
          } else {
            sum_post[k * V + t] += d[k][t] * m;
          }
          g[k][t] = du * gain;
          dot[0] = __builtin_fma((double)g[k][t], (double)m, dot[0]);
        }
      }
      float mean = 0.f;
      if (a.post) {
        row_total<G, 1, THREADS>(dot, buf[1]);
        mean = (float)(dot[0] * a.over);
      }
      if (a.dh) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int64_t j = (int64_t)(lane + G * k) * V, left = in ? a.D - j : 0;
#pragma unroll
          for (int t = 0; t < V; ++t) g[k][t] = r * (g[k][t] - h[k][t] * r * mean);
          store_columns<T, V>(a.dh + row * a.ld_dh + j, left, g[k]);
        }
      }
      if constexpr (GATES) {
        const int64_t g0 = gate_row * a.per_gate, g1 = g0 + a.per_gate;
        if (a.sums_gate && in && (row + 1 == g1 || row + 1 == end)) {
          const bool here = g0 >= first && g1 <= end;
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const int64_t j = (int64_t)(lane + G * k) * V, left = a.D - j;
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
          for (int e = 0; e < kEach; ++e) sum_gate[e] = 0.f;
        }
      }
    }
    if constexpr (G > 64) __syncthreads();
  }
  if (a.gain) columns_out<T, G, THREADS>(sum_gain, cols, a.partial + (int64_t)blockIdx.x * a.D, a.D);
  if (a.sums_post)
    columns_out<T, G, THREADS>(sum_post, cols, a.partial + ((int64_t)gridDim.x + blockIdx.x) * a.D, a.D);
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
  if (j < a.D)
    for (int32_t b = l; b < a.blocks; b += 8) v += p[b * a.D + j];
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

// Gate rows that reach over runs: their parts in order.  (No tokens: zeros.)
template <class G_>
__global__ void __launch_bounds__(256) k_gate_join(int64_t D, int64_t T_, int64_t rows, int64_t run, int64_t per_gate,
                                                   const float* partial, G_* dgate, int64_t ld, int32_t accumulate) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= D) return;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const int64_t g0 = row * per_gate, r0 = g0 / run, r1 = (g0 + per_gate - 1) / run;
    if (T_ && r0 == r1) continue;
    float v = 0.f;
    if (T_) {
#pragma unroll 8
      for (int64_t r = r0; r <= r1; ++r) v += partial[(r * 2 + (r == r0 ? 1 : 0)) * D + j];
    }
    G_* to = dgate + row * ld + j;
    *to = (G_)(accumulate ? (float)*to + v : v);
  }
}

// Threads per row, and of the workgroup in the backward.
int row_threads(int64_t D) { return D <= 256 ? 16 : D <= 1024 ? 64 : D <= 4096 ? 256 : 1024; }

// Runs of the backward: about one workgroup a compute unit, each row group
// with as few rows as that leaves.
constexpr int64_t kBlocks = 256;
struct Runs {
  int64_t rows, count, blocks;
  Runs(int64_t T, int64_t D) {
    const int64_t groups = 1024 / row_threads(D);
    rows = std::max<int64_t>(1, (T + kBlocks * groups - 1) / (kBlocks * groups));
    count = (T + rows - 1) / rows;
    blocks = std::max<int64_t>(1, (count + groups - 1) / groups);
  }
};

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
  auto launch = [&](auto kernel, int threads, int rows) {
    const int64_t blocks = std::min<int64_t>((l.T + rows - 1) / rows, (int64_t)1 << 20);
    kernel<<<dim3((uint32_t)blocks), threads, 0, stream>>>(a);
  };
  switch (row_threads(l.D)) {
    case 16: launch(k_norm<T, 16, 256>, 256, 16); break;
    case 64: launch(k_norm<T, 64, 256>, 256, 4); break;
    case 256: launch(k_norm<T, 256, 256>, 256, 1); break;
    default: launch(k_norm<T, 1024, 1024>, 1024, 1); break;
  }
  return hipGetLastError();
}

template <class T, class G_>
hipError_t norm_back(const NormLaunch& l, hipStream_t stream) {
  const Runs runs(l.T, l.D);
  const bool gates = l.gate && l.gate_rows > 1;
  NormBack<T, G_> a{};
  a.T_ = l.T;
  a.D = l.D;
  a.dy = static_cast<const T*>(l.dy);
  a.ds = static_cast<const T*>(l.ds);
  a.s = static_cast<const T*>(l.x);
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
  auto launch = [&](auto one, auto several, int threads) {
    if (gates) several<<<dim3((uint32_t)runs.blocks), threads, 0, stream>>>(a);
    else one<<<dim3((uint32_t)runs.blocks), threads, 0, stream>>>(a);
  };
  switch (row_threads(l.D)) {
    case 16: launch(k_norm_back<T, G_, 16, 1024, false>, k_norm_back<T, G_, 16, 1024, true>, 1024); break;
    case 64: launch(k_norm_back<T, G_, 64, 1024, false>, k_norm_back<T, G_, 64, 1024, true>, 1024); break;
    case 256: launch(k_norm_back<T, G_, 256, 1024, false>, k_norm_back<T, G_, 256, 1024, true>, 1024); break;
    default: launch(k_norm_back<T, G_, 1024, 1024, false>, k_norm_back<T, G_, 1024, 1024, true>, 1024); break;
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

int64_t norm_workspace(int64_t T, int64_t D, int64_t gate_rows) {
  const Runs runs(T, D);
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
