// The tile product under the linear layer and the Newton-Schulz steps:
//   C(i, j) = sum_k A(i, k) B(j, k)
// for one BM x BN tile of C, on the matrix cores, accumulated in fp32.
//
// Either operand may have k contiguous in memory (row i is a run of k: "KC")
// or k strided (row k is a run of i: "KS"), so x wT (KC, KC), dz w (KC, KS)
// and dzT x (KS, KS) are one kernel with nothing transposed in memory.
//
// A stage is 128 bytes of k per row (64 values of 16 bits, 32 of fp32).  Its
// 16-byte chunks are stored XOR-permuted so that the fragment reads of a wave
// spread over the LDS banks: a KC operand as [row][k], read with 16-byte
// reads; a KS operand as [k][row], read with the transposing 8-byte reads
// (16 bits) or 4-byte reads (fp32).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "internal.h"

namespace dc {

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));

// One k-slice of products: 32 values of k for the 16-bit types, 16 for fp32
// (four instructions of 4; the order of k inside a slice is the same for
// both operands and otherwise free).  D's row index runs over `b`'s rows, so
// a lane holds four neighbouring columns j of one row i.
__device__ __forceinline__ f32x4 mma_slice(u32x4 b, u32x4 a, f32x4 c, __bf16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c,
                                                 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma_slice(u32x4 b, u32x4 a, f32x4 c, _Float16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), c, 0,
                                                0, 0);
}
__device__ __forceinline__ f32x4 mma_slice(u32x4 b, u32x4 a, f32x4 c, float) {
#pragma unroll
  for (int t = 0; t < 4; ++t)
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(b[t]), __uint_as_float(a[t]), c, 0, 0, 0);
  return c;
}

// One operand of a tile: `p` is the first value of the tile's first row (KC)
// or column (KS), `rows` how many rows of the tile exist.
template <class T>
struct Operand {
  const T* p;
  int64_t ld;
  int32_t rows;
};

// ROWS rows of one operand: the addresses of its stage in LDS.
template <class T, int ROWS, bool KC>
struct StageMap {
  static constexpr int ES = sizeof(T);
  static constexpr int EPC = 16 / ES;                  // values per 16-byte chunk
  static constexpr int BK = 128 / ES;                  // values of k per stage
  static constexpr int CPR = KC ? 8 : ROWS / EPC;      // chunks per LDS row
  static constexpr int kChunks = ROWS * 8;
  static constexpr int kBytes = ROWS * 128;

  // The permutation of a row's chunks (an involution: XOR).
  __device__ static int swizzle(int line) {
    if constexpr (KC) return line & 7;
    else if constexpr (ES == 4) return ((line >> 2) & 3) << 2;
    else if constexpr (CPR >= 16) return ((line & 3) | (((line >> 3) & 1) << 2)) << 1;
    else return (((line >> 1) & 1) | (((line >> 3) & 1) << 1)) << 1;
  }

  // Fragment of 16 rows from `row0` for k-slice `ks`, for lane (q, r) =
  // (lane / 16, lane % 16): this lane's share of row row0 + r.
  __device__ static u32x4 fragment(const char* lds, int row0, int ks, int q, int r) {
    if constexpr (KC) {
      const int row = row0 + r;
      return *reinterpret_cast<const u32x4*>(lds + row * 128 + (((ks * 4 + q) ^ swizzle(row)) << 4));
    } else if constexpr (ES == 4) {
      u32x4 v;
      const int col = row0 + r;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int k = ks * 16 + q * 4 + t;
        v[t] = *reinterpret_cast<const uint32_t*>(lds + k * (CPR * 16) + (((col >> 2) ^ swizzle(k)) << 4) +
                                                  ((col & 3) << 2));
      }
      return v;
    } else {
      // The transposing read: the 16 lanes of a group name 16 runs of four
      // values, run 4 a + b = columns 4 b.. of row a, and lane r receives
      // column r of rows 0..3.
      u32x4 v;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = ks * 32 + q * 8 + h * 4 + (r >> 2);
        const int col = row0 + ((r & 3) << 2);
        const char* p = lds + k * (CPR * 16) + (((col >> 3) ^ swizzle(k)) << 4) + ((col & 4) << 1);
        const i16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) i16x4*)(p));
        const uint64_t u = __builtin_bit_cast(uint64_t, t);
        v[2 * h] = (uint32_t)u;
        v[2 * h + 1] = (uint32_t)(u >> 32);
      }
      return v;
    }
  }
};

// Loads through registers: any address and any size.  A chunk wholly inside
// is one 16-byte load (unaligned where the operand is); one that crosses the
// operand's end is read value by value, and what is outside counts as zero.
template <class T, int ROWS, bool KC, int NT>
struct RegisterLoader {
  using Map = StageMap<T, ROWS, KC>;
  static constexpr int kPer = Map::kChunks / NT;
  static_assert(Map::kChunks % NT == 0, "chunks divide over the threads");
  u32x4 v[kPer];

  __device__ void load(const Operand<T>& op, int64_t k0, int64_t k_end, int tid) {
#pragma unroll
    for (int s = 0; s < kPer; ++s) {
      const int c = s * NT + tid;
      const int line = c / Map::CPR, chunk = (c % Map::CPR) ^ Map::swizzle(line);
      int64_t left;
      const T* p;
      if constexpr (KC) {
        const int64_t k = k0 + chunk * Map::EPC;
        left = line < op.rows ? k_end - k : 0;
        p = op.p + (int64_t)line * op.ld + k;
      } else {
        const int64_t k = k0 + line;
        left = k < k_end ? op.rows - chunk * Map::EPC : 0;
        p = op.p + k * op.ld + chunk * Map::EPC;
      }
      u32x4 x = {0, 0, 0, 0};
      if (left >= Map::EPC) {
        __builtin_memcpy(&x, p, 16);
      } else if (left > 0) {
        T e[Map::EPC];
#pragma unroll
        for (int t = 0; t < Map::EPC; ++t) e[t] = t < left ? p[t] : (T)0;
        __builtin_memcpy(&x, e, 16);
      }
      v[s] = x;
    }
  }

  __device__ void store(char* lds, int tid) const {
#pragma unroll
    for (int s = 0; s < kPer; ++s) *reinterpret_cast<u32x4*>(lds + (s * NT + tid) * 16) = v[s];
  }
};

// One BM x BN tile by WM x WN waves; each wave holds MI x NI blocks of 16x16.
template <class T, int BM, int BN, int WM, int WN, bool KCA, bool KCB>
struct TileProduct {
  static constexpr int NT = WM * WN * 64;
  static constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  using MapA = StageMap<T, BM, KCA>;
  using MapB = StageMap<T, BN, KCB>;
  static constexpr int BK = MapA::BK;
  static constexpr int kLds = MapA::kBytes + MapB::kBytes;

  // acc += A B over k in [k0, k_end); lds holds kLds bytes, 16-byte aligned.
  __device__ static void run(const Operand<T>& a, const Operand<T>& b, int64_t k0, int64_t k_end, char* lds,
                             f32x4 (&acc)[MI][NI]) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int q = lane >> 4, r = lane & 15;
    const int row_a = (wave / WN) * (BM / WM), row_b = (wave % WN) * (BN / WN);
    char* la = lds;
    char* lb = lds + MapA::kBytes;
    RegisterLoader<T, BM, KCA, NT> ra;
    RegisterLoader<T, BN, KCB, NT> rb;
    ra.load(a, k0, k_end, tid);
    rb.load(b, k0, k_end, tid);
    for (; k0 < k_end; k0 += BK) {
      __syncthreads();  // every wave is done with the stage in LDS
      ra.store(la, tid);
      rb.store(lb, tid);
      __syncthreads();
      if (k0 + BK < k_end) {
        ra.load(a, k0 + BK, k_end, tid);
        rb.load(b, k0 + BK, k_end, tid);
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        u32x4 fa[MI], fb[NI];
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[i] = MapA::fragment(la, row_a + i * 16, ks, q, r);
#pragma unroll
        for (int j = 0; j < NI; ++j) fb[j] = MapB::fragment(lb, row_b + j * 16, ks, q, r);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < NI; ++j) acc[i][j] = mma_slice(fb[j], fa[i], acc[i][j], T{});
      }
    }
  }

  // f(i, j, v): rows and columns inside the tile, v the sums of columns
  // j .. j + 3 of row i.
  template <class F>
  __device__ static void each(const f32x4 (&acc)[MI][NI], F&& f) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row_a = (wave / WN) * (BM / WM) + (lane & 15), row_b = (wave % WN) * (BN / WN) + (lane >> 4) * 4;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) f(row_a + i * 16, row_b + j * 16, acc[i][j]);
  }
};

// Four neighbouring values of a row as fp32, and back; `n` of them exist
// (at least one).  The whole group is one access, unaligned where the row is.
template <class T>
__device__ __forceinline__ f32x4 load4(const T* p, int n) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (n >= 4) {
    T e[4];
    __builtin_memcpy(e, p, sizeof e);
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = (float)e[t];
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (t < n) v[t] = (float)p[t];
  }
  return v;
}

template <class T>
__device__ __forceinline__ void store4(T* p, f32x4 v, int n) {
  if (n >= 4) {
    T e[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) e[t] = (T)v[t];
    __builtin_memcpy(p, e, sizeof e);
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (t < n) p[t] = (T)v[t];
  }
}

// Workgroup b of n, with the workgroups of one XCD (b mod 8) on one run of
// consecutive tiles, so that neighbouring tiles share operands in its L2.
__device__ __forceinline__ int64_t xcd_run(int64_t b, int64_t n) { return tile_slot(b, n); }

// Tile t of a rows x cols grid, walked in bands of `band` tile rows.
__device__ __forceinline__ void band_tile(int64_t t, int64_t rows, int64_t cols, int band, int64_t& ti, int64_t& tj) {
  const int64_t per = (int64_t)band * cols;
  const int64_t g = t / per, first = g * band;
  const int64_t h = rows - first < band ? rows - first : band;
  const int64_t in = t - g * per;
  ti = first + in % h;
  tj = in / h;
}

}  // namespace dc
