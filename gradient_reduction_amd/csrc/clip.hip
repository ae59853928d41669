// The global norm over a list of gradients, and clipping by it:
//   n = sqrt(sum of every element's square),  c = min(1, max_norm / (n + eps)),  out = c grad
// Squares and their sums are fp64: fp32 gradients of any size neither overflow
// nor vanish, and the order of the sum is fixed by the sizes alone.
//
// Gradients are cut into units of 16 KB.  A launch's list travels as kernel
// arguments, flat gradients (one run of elements) and strided ones apart; its
// workgroups take units in turn and keep their place in the list.
//
// Bound by the bytes: 2 GiB of fp32 or bf16 are read at 5.9 TB/s; 100M bf16
// take 34 us and 66 more to be scaled (6.1 TB/s read and written); 395M fp32
// 840 in all, 5.6 TB/s.  Units of 8 and 32 KB took 4% and 6% more on those.
// 113 vectors: 5.5 and 5.3 us.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "columns.h"
#include "device_common.h"
#include "internal.h"

namespace dc {
namespace {

constexpr int64_t kUnit = 16384;      // bytes
constexpr int64_t kLaunchUnits = (int64_t)1 << 30;

// Flat gradients of one launch: numel2 = 2 numel + (fp32).
struct FlatList {
  static constexpr int kMost = 140;
  int32_t count;
  const void* grad[kMost];
  void* out[kMost];
  int64_t numel2[kMost];
  int32_t begin[kMost + 1];  // first unit
};

// Strided ones.
struct RowsList {
  static constexpr int kMost = 64;
  int32_t count;
  const void* grad[kMost];
  void* out[kMost];
  int64_t ld_grad[kMost], ld_out[kMost];
  int64_t cols2[kMost];
  int32_t row_units[kMost];
  int32_t begin[kMost + 1];
};
static_assert(sizeof(FlatList) + 96 <= 4096 && sizeof(RowsList) + 96 <= 4096, "kernel arguments");

// One unit: n elements, fp32 or bf16.
struct Unit {
  const char* grad;
  char* out;
  int32_t n;
  bool wide;
};

__device__ __forceinline__ Unit unit_at(const FlatList& l, int e, int32_t u) {
  Unit t;
  t.wide = l.numel2[e] & 1;
  const int64_t per = t.wide ? kUnit / 4 : kUnit / 2, numel = l.numel2[e] >> 1;
  const int64_t at = (int64_t)(u - l.begin[e]) * kUnit, left = numel - (int64_t)(u - l.begin[e]) * per;
  t.grad = static_cast<const char*>(l.grad[e]) + at;
  t.out = static_cast<char*>(l.out[e]) + at;
  t.n = (int32_t)(left < per ? left : per);
  return t;
}

__device__ __forceinline__ Unit unit_at(const RowsList& l, int e, int32_t u) {
  Unit t;
  t.wide = l.cols2[e] & 1;
  const int32_t es = t.wide ? 4 : 2;
  const int64_t per = kUnit / es, cols = l.cols2[e] >> 1;
  const int32_t k = u - l.begin[e];
  const int64_t row = k / l.row_units[e], at = (int64_t)(k % l.row_units[e]) * per, left = cols - at;
  t.grad = static_cast<const char*>(l.grad[e]) + (row * l.ld_grad[e] + at) * es;
  t.out = static_cast<char*>(l.out[e]) + (row * l.ld_out[e] + at) * es;
  t.n = (int32_t)(left < per ? left : per);
  return t;
}

// The sum of v over a workgroup of 256, to every thread.
__device__ __forceinline__ double group_total(double v) {
  __shared__ double part[4];
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

// A unit's elements in 16-byte vectors, four to a thread; the last of them may
// be short.
constexpr int kVectors = kUnit / 16 / 256;

__device__ __forceinline__ u32x4 load_part(const char* p, int have, bool wide) {
  u32x4 v = {0, 0, 0, 0};
  if (wide) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (t < have) v[t] = reinterpret_cast<const uint32_t*>(p)[t];
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (t < have) v[t / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[t] << (16 * (t & 1));
  }
  return v;
}

// Vectors of a unit: elements past its end read as zeros.
__device__ __forceinline__ void load_unit(const Unit& t, bool streamed, u32x4 (&v)[kVectors]) {
  const int V = t.wide ? 4 : 8;
  if (t.n == kVectors * 256 * V) {
#pragma unroll
    for (int j = 0; j < kVectors; ++j) {
      const u32x4_any* p = reinterpret_cast<const u32x4_any*>(t.grad + 16 * (j * 256 + (int)threadIdx.x));
      if (streamed) v[j] = __builtin_nontemporal_load(p);
      else v[j] = *p;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kVectors; ++j) {
    const int i = j * 256 + (int)threadIdx.x, have = t.n - i * V;
    if (have >= V) v[j] = *reinterpret_cast<const u32x4_any*>(t.grad + 16 * i);
    else v[j] = have > 0 ? load_part(t.grad + 16 * i, have, t.wide) : u32x4{0, 0, 0, 0};
  }
}

// The entry of unit u: every lane looks at one in 64 of the list's beginnings,
// so that a long list costs one read of the arguments, not one per entry.
template <class List>
__device__ __forceinline__ int find_entry(const List& l, int32_t u) {
  int n = 0;
#pragma unroll
  for (int k = 0; k < List::kMost; k += 64) {
    const int e = k + (threadIdx.x & 63);
    n += __popcll(__ballot(e < l.count && l.begin[e] <= u));
  }
  return __builtin_amdgcn_readfirstlane(n - 1);
}

// The squares are summed from the list's beginning to its end and the
// gradients scaled from its end to its beginning: what was read last is then
// still in the 256 MB cache.  Units further than kCached from the end are
// streamed both times, past what is kept: 100M bf16 118 to 103 us, 395M fp32 889
// to 844.  (How much of the second read the cache serves was not measured; a
// copy of as many bytes from HBM takes 59 of the 66 us.)
constexpr int64_t kCached = ((int64_t)192 << 20) / kUnit;

// partial[workgroup] (+)= the squares of its units.  `after`: units that later
// launches read.
template <class List>
__global__ void __launch_bounds__(256) k_squares(List l, int64_t after, double* partial, int32_t add) {
  double s = 0;
  const int32_t units = l.begin[l.count];
  int e = (int32_t)blockIdx.x < units ? find_entry(l, blockIdx.x) : 0;
  for (int32_t u = blockIdx.x; u < units; u += gridDim.x) {
    while (l.begin[e + 1] <= u) ++e;
    const Unit t = unit_at(l, e, u);
    u32x4 v[kVectors];
    load_unit(t, after + units - u > kCached, v);
#pragma unroll
    for (int j = 0; j < kVectors; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (t.wide) {
          const double a = __uint_as_float(v[j][q]);
          s = __builtin_fma(a, a, s);
        } else {
          const double a = bf16_lo(v[j][q]), b = bf16_hi(v[j][q]);
          s = __builtin_fma(a, a, s);
          s = __builtin_fma(b, b, s);
        }
      }
  }
  s = group_total(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = add ? partial[blockIdx.x] + s : s;
}

__device__ __forceinline__ double fold_partials(const double* partial, int32_t parts) {
  double s = 0;
  for (int32_t i = threadIdx.x; i < parts; i += 256) s += partial[i];
  return group_total(s);
}

__global__ void __launch_bounds__(256) k_norm(const double* partial, int32_t parts, int32_t add, double* squares,
                                              float* norm) {
  double s = fold_partials(partial, parts);
  if (threadIdx.x) return;
  if (squares) {
    if (add) s += *squares;
    *squares = s;
  }
  if (norm) *norm = (float)sqrt(s);
}

// The factor: 1 unless the norm passes max_norm; a NaN norm gives NaN.
__device__ __forceinline__ float factor(double squares, float max_norm, float eps) {
  const double n = sqrt(squares) + (double)eps;
  return n <= (double)max_norm ? 1.f : (float)((double)max_norm / n);
}

// Every workgroup folds the partial sums by itself (16 KB from the caches) or
// takes the given sum, then scales its units.  The list has the gradients in
// reverse order, and each is gone through from its end.  `before`: units of
// earlier launches.  A factor of 1 leaves nothing to do in place (in_place: the
// whole list is).
template <class List>
__global__ void __launch_bounds__(256) k_clip(List l, int64_t before, const double* partial, int32_t parts,
                                              const double* squares, float max_norm, float eps, float* norm,
                                              float* coef, int32_t in_place) {
  const double s = squares ? *squares : fold_partials(partial, parts);
  const float c = factor(s, max_norm, eps);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (norm) *norm = (float)sqrt(s);
    if (coef) *coef = c;
  }
  if (in_place && c == 1.f) return;
  const int32_t units = l.begin[l.count];
  int e = (int32_t)blockIdx.x < units ? find_entry(l, blockIdx.x) : 0;
  for (int32_t u = blockIdx.x; u < units; u += gridDim.x) {
    while (l.begin[e + 1] <= u) ++e;
    const Unit t = unit_at(l, e, l.begin[e] + l.begin[e + 1] - 1 - u);
    if (t.out == t.grad && c == 1.f) continue;
    u32x4 v[kVectors];
    load_unit(t, before + u > kCached, v);
    const int V = t.wide ? 4 : 8;
#pragma unroll
    for (int j = 0; j < kVectors; ++j) {
      const int i = j * 256 + (int)threadIdx.x, have = t.n - i * V;
      if (have <= 0) continue;
      u32x4 y;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (t.wide) y[q] = __float_as_uint(c * __uint_as_float(v[j][q]));
        else y[q] = bf16_pack_out(c * bf16_lo(v[j][q]), c * bf16_hi(v[j][q]));
      }
      char* to = t.out + 16 * i;
      if (have >= V) {
        __builtin_nontemporal_store((u32x4_any)y, reinterpret_cast<u32x4_any*>(to));
      } else if (t.wide) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q < have) reinterpret_cast<uint32_t*>(to)[q] = y[q];
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < have) reinterpret_cast<uint16_t*>(to)[q] = (uint16_t)(y[q / 2] >> (16 * (q & 1)));
      }
    }
  }
}

// Calls f(list, units, units of the launches before) for every launch's part of
// the gradients, in reverse order where they are written.  `rows`: of a
// gradient, how many take part.
template <class Rows, class F>
void for_lists(const dc_gradient* grads, int32_t num, Rows rows, bool writes, F&& f) {
  int64_t before = 0;
  FlatList flat;
  RowsList strided;
  flat.count = strided.count = 0;
  flat.begin[0] = strided.begin[0] = 0;
  auto close = [&](auto& l) {
    if (l.count) {
      f(l, l.begin[l.count], before);
      before += l.begin[l.count];
    }
    l.count = 0;
  };
  auto units = [&](auto& l, int64_t n) {  // of a new entry; true: it fits
    if (l.count == l.kMost || l.begin[l.count] + n > kLaunchUnits) close(l);
    l.begin[l.count + 1] = l.begin[l.count] + (int32_t)n;
    return l.count++;
  };
  for (int32_t k = 0; k < num; ++k) {
    const dc_gradient& g = grads[writes ? num - 1 - k : k];
    const int64_t r = rows(g), es = g.dtype == DC_F32 ? 4 : 2, per = kUnit / es;
    if (r == 0 || g.cols == 0) continue;
    if (r == 1 || (g.ld_grad == g.cols && (!writes || g.ld_out == g.cols))) {
      const int64_t n = r * g.cols;
      const int32_t i = units(flat, (n + per - 1) / per);
      flat.grad[i] = g.grad;
      flat.out[i] = g.out;
      flat.numel2[i] = 2 * n + (g.dtype == DC_F32);
      continue;
    }
    // rows in runs that one launch's units hold
    const int64_t ru = (g.cols + per - 1) / per, most = kLaunchUnits / ru;
    for (int64_t r0 = 0; r0 < r; r0 += most) {
      const int32_t i = units(strided, std::min(most, r - r0) * ru);
      strided.grad[i] = static_cast<const char*>(g.grad) + r0 * g.ld_grad * es;
      strided.out[i] = writes ? static_cast<char*>(g.out) + r0 * g.ld_out * es : nullptr;
      strided.ld_grad[i] = g.ld_grad;
      strided.ld_out[i] = g.ld_out;
      strided.cols2[i] = 2 * g.cols + (g.dtype == DC_F32);
      strided.row_units[i] = (int32_t)ru;
    }
  }
  close(flat);
  close(strided);
}

// Workgroups of a launch: eight of 256 threads a compute unit, 2048 in all,
// hold every wave that fits, and their sums are 16 KB.
constexpr int32_t kParts = 2048;

struct Counted {
  int32_t parts;
  int64_t units;
};
Counted counted(const dc_gradient* grads, int32_t num) {
  Counted c{1, 0};
  for_lists(grads, num, [](const dc_gradient& g) { return g.counted; }, false,
            [&](const auto&, int32_t units, int64_t) {
              c.parts = std::max(c.parts, std::min(units, kParts));
              c.units += units;
            });
  return c;
}

void sum_squares(const dc_gradient* grads, int32_t num, const Counted& c, double* partial, hipStream_t stream) {
  const dim3 grid((uint32_t)c.parts);
  for_lists(grads, num, [](const dc_gradient& g) { return g.counted; }, false,
            [&](const auto& l, int32_t units, int64_t before) {
              k_squares<<<grid, 256, 0, stream>>>(l, c.units - before - units, partial, before > 0);
            });
  if (c.units == 0) {  // nothing is counted
    FlatList none;
    none.count = 0;
    none.begin[0] = 0;
    k_squares<<<grid, 256, 0, stream>>>(none, (int64_t)0, partial, 0);
  }
}

}  // namespace

int64_t clip_workspace() { return kParts * 8; }

hipError_t launch_grad_norm(const dc_gradient* grads, int32_t num, int32_t accumulate, double* squares, float* norm,
                            void* workspace, hipStream_t stream) {
  double* partial = static_cast<double*>(workspace);
  const Counted c = counted(grads, num);
  sum_squares(grads, num, c, partial, stream);
  k_norm<<<1, 256, 0, stream>>>(partial, c.parts, accumulate, squares, norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const dc_gradient* grads, int32_t num, const double* squares, float max_norm, float eps,
                            float* norm, float* coef, void* workspace, hipStream_t stream) {
  double* partial = static_cast<double*>(workspace);
  int32_t parts = 0, in_place = 1, launches = 0;
  if (!squares) {
    const Counted c = counted(grads, num);
    sum_squares(grads, num, c, partial, stream);
    parts = c.parts;
  }
  for (int32_t k = 0; k < num; ++k) in_place &= grads[k].out == grads[k].grad;
  auto clip = [&](const auto& l, int32_t units, int64_t before) {
    k_clip<<<dim3((uint32_t)std::max(1, std::min(units, kParts))), 256, 0, stream>>>(
        l, before, partial, parts, squares, max_norm, eps, norm, coef, in_place);
    ++launches;
  };
  for_lists(grads, num, [](const dc_gradient& g) { return g.rows; }, true, clip);
  if (!launches) {  // no elements: the norm and the factor alone
    FlatList none;
    none.count = 0;
    none.begin[0] = 0;
    clip(none, 0, 0);
  }
  return hipGetLastError();
}

}  // namespace dc
