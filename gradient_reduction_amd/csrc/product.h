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

#include <type_traits>
#include <utility>

#include "device_common.h"
#include "internal.h"

namespace dc {

typedef float f32x8 __attribute__((ext_vector_type(8)));
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

typedef __attribute__((address_space(3))) char* LdsPtr;

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

  // Where lane (q, r) = (lane / 16, lane % 16) finds its share of the 16-row
  // fragments of rows row0, row0 + 16, ..: row0 is a multiple of all the
  // fragments' rows.  The permutation depends on the lane alone, so fragment
  // i and k-slice ks are reached from here by an XOR or a constant offset.
  __device__ static uint32_t lane_base(int row0, int q, int r) {
    if constexpr (KC) {
      return (row0 + r) * 128 + ((q ^ swizzle(r)) << 4);
    } else if constexpr (ES == 4) {
      return q * 4 * (CPR * 16) + ((((row0 + r) >> 2) ^ swizzle(q * 4)) << 4) + ((r & 3) << 2);
    } else {
      const int k = q * 8 + (r >> 2), col = row0 + ((r & 3) << 2);
      return k * (CPR * 16) + (((col >> 3) ^ swizzle(k)) << 4) + ((col & 4) << 1);
    }
  }

  __device__ static u32x4 fragment(LdsPtr lds, uint32_t base, int i, int ks) {
    if constexpr (KC) {
      return *(const __attribute__((address_space(3))) u32x4*)(lds + (base ^ (ks << 6)) + i * 2048);
    } else if constexpr (ES == 4) {
      u32x4 v;
#pragma unroll
      for (int t = 0; t < 4; ++t)
        v[t] = *(const __attribute__((address_space(3))) uint32_t*)(lds + (base ^ (i << 6)) +
                                                                    (ks * 16 + t) * (CPR * 16));
      return v;
    } else {
      // The transposing read: the 16 lanes of a group name 16 runs of four
      // values, run 4 a + b = columns 4 b.. of row a, and lane r receives
      // column r of rows 0..3.
      u32x4 v;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const i16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) i16x4*)(lds + (base ^ (i << 5)) + (ks * 32 + h * 4) * (CPR * 16)));
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
// A whole stage is loaded with no condition for each chunk: rows (columns, of
// a KS operand) outside only make sums that nobody writes, so they get the
// values of a row inside, and a KS chunk across a row's end takes in the next
// row's beginning, which exists in all stages but the last.
template <class T, int ROWS, bool KC, int NT>
struct RegisterLoader {
  using Map = StageMap<T, ROWS, KC>;
  static constexpr int kPer = Map::kChunks / NT;
  static_assert(Map::kChunks % NT == 0, "chunks divide over the threads");
  u32x4 v[kPer];

  __device__ void load(const Operand<T>& op, int64_t k0, int64_t k_end, int tid) {
    if (KC ? k0 + Map::BK <= k_end : k0 + Map::BK < k_end && op.ld >= Map::EPC) {
      const T* base = op.p + (KC ? k0 : k0 * op.ld);
#pragma unroll
      for (int s = 0; s < kPer; ++s) {
        const int c = s * NT + tid;
        const int line = c / Map::CPR, chunk = (c % Map::CPR) ^ Map::swizzle(line);
        const int row = KC && line >= op.rows ? 0 : line;
        const int at = !KC && chunk * Map::EPC >= op.rows ? 0 : chunk * Map::EPC;
        __builtin_memcpy(&v[s], base + row * op.ld + at, 16);
      }
      return;
    }
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

// Loads straight into LDS, for operands whose chunks are whole and aligned
// (see direct_operand): a wave's 64 chunks land behind each other, so the
// permutation is applied to the addresses they come from.  What is outside
// gets an offset past the resource's end and arrives as zero.
template <class T, int ROWS, bool KC, int NT>
struct DirectLoader {
  using Map = StageMap<T, ROWS, KC>;
  static constexpr int kPer = Map::kChunks / NT;
  static constexpr uint32_t kOutside = 0x80000000u;
  uint32_t offset[kPer], last[kPer];  // of whole stages, and of one of `rest` values of k

  __device__ void init(const Operand<T>& op, int rest, int tid) {
#pragma unroll
    for (int s = 0; s < kPer; ++s) {
      const int c = s * NT + tid;
      const int line = c / Map::CPR, chunk = (c % Map::CPR) ^ Map::swizzle(line);
      const bool in = KC ? line < op.rows : chunk * Map::EPC < op.rows;
      offset[s] = in ? (uint32_t)line * (uint32_t)(op.ld * Map::ES) + chunk * 16 : kOutside;
      last[s] = (KC ? chunk * Map::EPC : line) < rest ? offset[s] : kOutside;
    }
  }

  // The stage at k0 into lds; `left` = k_end - k0.  One past the end reads
  // nothing (its resource is empty).
  __device__ void load(const Operand<T>& op, int64_t k0, int64_t left, char* lds, int wave) const {
    const T* base = op.p + (KC ? k0 : k0 * op.ld);
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<T*>(base), (short)0, left > 0 ? (int)kOutside : 0, kBufferFlags);
    const bool whole = left >= Map::BK;
#pragma unroll
    for (int s = 0; s < kPer; ++s)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, (__attribute__((address_space(3))) void*)(lds + (s * NT + wave * 64) * 16), 16,
          (int)(whole ? offset[s] : last[s]), 0, 0, 0);
  }
};

// Whether a stage of `op`'s matrix can be loaded straight into LDS: 16-byte
// rows, contiguous lengths of whole chunks, and offsets inside a tile under
// 2^31 bytes.
template <class T>
inline bool direct_operand(const void* p, int64_t ld, int64_t contiguous) {
  constexpr int64_t epc = 16 / sizeof(T);
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % epc == 0 && contiguous % epc == 0 &&
         ld * (int64_t)sizeof(T) * 256 < ((int64_t)1 << 31);
}

// One BM x BN tile by WM x WN waves; each wave holds MI x NI blocks of 16x16.
// A stage's memory: one variable per stage, so that the compiler sees that
// reading one does not wait for what is arriving in another.
template <int I, int BYTES>
__device__ __forceinline__ char* stage_memory() {
  __shared__ __attribute__((aligned(16))) char memory[BYTES];
  return memory;
}

template <class F, int... I>
__device__ __forceinline__ void each_index(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}

// S stages are in flight or being multiplied; loads through registers use one.
template <class T, int BM, int BN, int WM, int WN, bool KCA, bool KCB, int S>
struct TileProduct {
  static constexpr int NT = WM * WN * 64;
  static constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  using MapA = StageMap<T, BM, KCA>;
  using MapB = StageMap<T, BN, KCB>;
  static constexpr int BK = MapA::BK;
  static constexpr int kStage = MapA::kBytes + MapB::kBytes;
  static constexpr bool kDirect = S > 1;

  template <int I>
  __device__ static char* memory() { return stage_memory<I % S, kStage>(); }

  __device__ static void slice(LdsPtr la, LdsPtr lb, int ks, uint32_t base_a, uint32_t base_b,
                               f32x4 (&acc)[MI][NI]) {
    u32x4 fa[MI], fb[NI];
#pragma unroll
    for (int j = 0; j < NI; ++j) fb[j] = MapB::fragment(lb, base_b, j, ks);
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[i] = MapA::fragment(la, base_a, i, ks);
    // All reads first: left to the compiler they trickle between the products,
    // with fewer in flight (8192^3 when it was chosen: 1115, 1270 and 1215
    // TFLOP/s for the three kinds of product; 1140, 1340 and 1310 so).
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = mma_slice(fb[j], fa[i], acc[i][j], T{});
  }

  // acc(i, j) += coef B(j, i) for the rows i of the tile (its first row being k
  // = i0) that the stage at k0 holds as its k: an operand that is also added
  // to the result is taken from the stage in LDS, not read again.  A wave's
  // rows are all in one stage.
  __device__ static void add_b(LdsPtr la, int64_t k0, int64_t i0, float coef, f32x4 (&acc)[MI][NI]) {
    static_assert(64 % (BM / WM) == 0 && sizeof(T) == 2, "stages hold whole waves' rows");
    typedef T V __attribute__((ext_vector_type(4)));
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, r = lane & 15;
    const int row_a = (wave / WN) * (BM / WM), row_b = (wave % WN) * (BN / WN);
    if (k0 != i0 + row_a / BK * BK) return;
    const LdsPtr lb = la + MapA::kBytes;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        V v;
        if constexpr (KCB) {  // rows j in LDS: read transposed, lane r its column r
          const int row = row_b + j * 16 + q * 4 + (r >> 2), k = row_a % BK + i * 16 + ((r & 3) << 2);
          v = __builtin_bit_cast(V, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                        (__attribute__((address_space(3))) i16x4*)(
                                            lb + row * 128 + (((k >> 3) ^ MapB::swizzle(row)) << 4) + ((k & 4) << 1))));
        } else {
          const int k = row_a % BK + i * 16 + r, col = row_b + j * 16 + q * 4;
          v = *(const __attribute__((address_space(3))) V*)(
              lb + k * (MapB::CPR * 16) + (((col >> 3) ^ MapB::swizzle(k)) << 4) + ((col & 4) << 1));
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[i][j][t] = fmaf(coef, (float)v[t], acc[i][j][t]);
      }
  }

  struct NoHook {
    __device__ void operator()(LdsPtr, int64_t) const {}
  };

  // acc += A B over k in [k0, k_end).  hook(la, k) is called when the stage of
  // k .. k + 63 is at la (loads straight into LDS only).
  template <class Hook = NoHook>
  __device__ static void run(const Operand<T>& a, const Operand<T>& b, int64_t k0, int64_t k_end,
                             f32x4 (&acc)[MI][NI], Hook&& hook = {}) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, r = lane & 15;
    const uint32_t base_a = MapA::lane_base((wave / WN) * (BM / WM), q, r);
    const uint32_t base_b = MapB::lane_base((wave % WN) * (BN / WN), q, r);
    if constexpr (kDirect) {
      __syncthreads();  // a product before this one is done with the stages
      DirectLoader<T, BM, KCA, NT> da;
      DirectLoader<T, BN, KCB, NT> db;
      const int rest = (int)((k_end - k0) % BK);
      da.init(a, rest, tid);
      db.init(b, rest, tid);
      // Stages past the end are loaded too, which reads nothing and keeps the
      // count of loads in flight the same.
      auto load = [&](char* to, int64_t k) {
        da.load(a, k, k_end - k, to, wave);
        db.load(b, k, k_end - k, to + MapA::kBytes, wave);
      };
      constexpr int kFlight = (S - 2) * (da.kPer + db.kPer);
      constexpr int kWait = (kFlight & 15) | (7 << 4) | ((kFlight >> 4) << 14);
      auto stage = [&](char* cur, char* last) {
        // this wave's part of the stage is there, and its reads of the one
        // before are done; then everybody's
        __builtin_amdgcn_s_waitcnt(kWait);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        load(last, k0 + (S - 1) * BK);
        __builtin_amdgcn_sched_barrier(0);  // the loads go out first (left to the end: 15% slower)
        const LdsPtr la = (LdsPtr)cur;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) slice(la, la + MapA::kBytes, ks, base_a, base_b, acc);
        hook(la, k0);
        k0 += BK;
      };
      each_index([&](auto i) { load(memory<i.value>(), k0 + i.value * BK); },
                 std::make_integer_sequence<int, S - 1>{});
      while (k0 < k_end)
        each_index(
            [&](auto i) {
              if (i.value == 0 || k0 < k_end) stage(memory<i.value>(), memory<i.value + S - 1>());
            },
            std::make_integer_sequence<int, S>{});
      __builtin_amdgcn_s_waitcnt(0x0f70);  // nothing arrives any more
    } else {
      // kAhead stages are on their way into registers: with one, a stage of a
      // 64 tile took 1.4 us, most of it waiting.
      constexpr int kAhead = BM <= 64 ? 4 : BM <= 128 ? 2 : 1;
      RegisterLoader<T, BM, KCA, NT> ra[kAhead];
      RegisterLoader<T, BN, KCB, NT> rb[kAhead];
      char* lds = memory<0>();
      const LdsPtr la = (LdsPtr)lds;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {  // past the end: zeros, nothing read
        ra[i].load(a, k0 + i * BK, k_end, tid);
        rb[i].load(b, k0 + i * BK, k_end, tid);
      }
      while (k0 < k_end) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (i > 0 && k0 >= k_end) break;
          __syncthreads();  // every wave is done with the stage in LDS
          ra[i].store(lds, tid);
          rb[i].store(lds + MapA::kBytes, tid);
          __syncthreads();
          ra[i].load(a, k0 + kAhead * BK, k_end, tid);
          rb[i].load(b, k0 + kAhead * BK, k_end, tid);
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) slice(la, la + MapA::kBytes, ks, base_a, base_b, acc);
          k0 += BK;
        }
      }
    }
  }

  // Hands the tile out eight values at a time: f(i, j, v) gets columns
  // j .. j + 7 of row i when `rows` is set and returns what it made of them;
  // ft(j, i, v) gets rows i .. i + 7 of column j when `cols` is (what f
  // returned, if both are), all inside the tile.  The accumulators go
  // through the stages' memory, each wave by itself, so that a wave's accesses
  // to the result are runs of whole rows (or columns) and the code for eight
  // values exists once: with it in place for every accumulator, an epilogue
  // with an activation no longer fitted the instruction cache and took ten
  // times the product.
  template <class F, class FT>
  __device__ static void each(const f32x4 (&acc)[MI][NI], bool rows, bool cols, F&& f, FT&& ft) {
    constexpr int WR = BM / WM, WC = BN / WN;
    constexpr int kShare = (WM * WN + S - 1) / S;  // waves per stage's memory
    constexpr int kWave = kStage / kShare;
    constexpr int kFit = kWave / (WC * 4);
    constexpr int RP = kFit >= WR ? WR : kFit >= WR / 2 ? WR / 2 : WR / 4;  // rows per pass
    static_assert(RP % 16 == 0 && RP <= kFit, "passes");
    constexpr int kMask = WC / 4 - 1;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, r = lane & 15;
    const int row0 = (wave / WN) * WR, col0 = (wave % WN) * WC;
    char* own = memory<0>();
    each_index(
        [&](auto i) {
          if (wave / kShare == i.value) own = memory<i.value>();
        },
        std::make_integer_sequence<int, S>{});
    const LdsPtr mem = (LdsPtr)own + (wave % kShare) * kWave;
    auto chunk = [&](int row, int c) { return mem + row * (WC * 4) + ((c ^ (row & kMask)) << 4); };
    __syncthreads();  // every wave is done with the last stage
#pragma unroll
    for (int p = 0; p < WR; p += RP) {
#pragma unroll
      for (int i = 0; i < RP / 16; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
          *(__attribute__((address_space(3))) f32x4*)chunk(i * 16 + r, j * 4 + q) = acc[p / 16 + i][j];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (rows) {
        constexpr int kLanes = WC / 8;
#pragma unroll 1
        for (int k = lane / kLanes; k < RP; k += 64 / kLanes) {
          const int c = (lane % kLanes) * 2;
          const f32x4 lo = *(const __attribute__((address_space(3))) f32x4*)chunk(k, c);
          const f32x4 hi = *(const __attribute__((address_space(3))) f32x4*)chunk(k, c + 1);
          const f32x8 v = f(row0 + p + k, col0 + c * 4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
          if (cols) {
            *(__attribute__((address_space(3))) f32x4*)chunk(k, c) = __builtin_shufflevector(v, v, 0, 1, 2, 3);
            *(__attribute__((address_space(3))) f32x4*)chunk(k, c + 1) = __builtin_shufflevector(v, v, 4, 5, 6, 7);
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
      if (cols) {
        constexpr int kLanes = RP / 8;
#pragma unroll 1
        for (int c = lane / kLanes; c < WC; c += 64 / kLanes) {
          const int k = (lane % kLanes) * 8;
          f32x8 v;
#pragma unroll
          for (int t = 0; t < 8; ++t)
            v[t] = *(const __attribute__((address_space(3))) float*)(chunk(k + t, c >> 2) + ((c & 3) << 2));
          ft(col0 + c, row0 + p + k, v);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
};

// N neighbouring values of a row as fp32, and back; `n` of them exist (at
// least one).  A whole group is one access (16 bytes at most), unaligned where
// the row is.
template <int N, class T>
__device__ __forceinline__ auto load_n(const T* p, int64_t n) {
  typedef float V __attribute__((ext_vector_type(N)));
  V v = (V)(0.f);
  if (n >= N) {
    T e[N];
    __builtin_memcpy(e, p, sizeof e);
#pragma unroll
    for (int t = 0; t < N; ++t) v[t] = (float)e[t];
  } else {
#pragma unroll
    for (int t = 0; t < N; ++t)
      if (t < n) v[t] = (float)p[t];
  }
  return v;
}

template <int N, class T, class V>
__device__ __forceinline__ void store_n(T* p, V v, int64_t n) {
  if (n >= N) {
    T e[N];
#pragma unroll
    for (int t = 0; t < N; ++t) e[t] = (T)v[t];
    __builtin_memcpy(p, e, sizeof e);
  } else {
#pragma unroll
    for (int t = 0; t < N; ++t)
      if (t < n) p[t] = (T)v[t];
  }
}

constexpr int64_t kComputeUnits = 256;

// Whether 128 tiles take four stages instead of two: with no more tiles than
// compute units each has a unit's memory for itself (2048 x 1024 over 4096
// bf16: 31.5 against 32.7 us forward, 26.5 against 28.2 us dw).  64 tiles keep
// three: with eight, the longer code costs what the depth hides (one 1024 x
// 1024 matrix orthogonalised: 173 us against 165).
inline bool deep_launch(int64_t tiles) { return tiles <= kComputeUnits; }

// Stages of a launch of `tiles` tiles whose operands are loaded straight into
// LDS.
inline int32_t launch_stages(int32_t tile, int64_t tiles) {
  return tile == 256 ? 2 : tile == 64 ? 3 : deep_launch(tiles) ? 4 : 2;
}

// Microseconds that a compute unit takes for a stage of a tile, as measured
// with the unit busy (one 256 tile, two of 128, three of 64 resident): 2
// tile^2 64 operations at 1.26, 1.0 and 0.55 PFLOP/s over the chip; fp32 is
// held by the matrix cores' fp32 rate.
inline double stage_us(bool f32, int tile) {
  if (f32) return tile == 256 ? 6.9 : tile == 128 ? 1.75 : 0.45;
  return tile == 256 ? 1.6 : tile == 128 ? 0.54 : 0.25;
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
