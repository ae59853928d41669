// An embedding's lookup with scaling, and its table's gradient by sorted tokens:
//   out[t] = scale E[ids[t]]                       (zeros for an id outside the table)
//   dE[v] (+)= scale sum over {t: ids[t] = v} of dy[t]
// The gradient's tokens are sorted by id, stably, so that every row's sum runs
// over ascending t: no atomics, the same result every time.  The sorted
// tokens are cut into tiles of 8 to 32; a wave adds up one tile's rows over one
// run of columns and writes every row of dE that lies whole in its tile.  A
// row whose tokens reach over tiles leaves one partial sum in each, which a
// second launch adds up in order; a frequent token is so spread over the chip.
//
// The sort is a least-significant-digit radix sort with ranks from ballots.
//
// 32768 tokens of a natural text's frequencies in a table of 151936 x 1024,
// bf16 added to fp32: sort 22 us (two passes, each of a count and a pass),
// rows 30 (167 MB, 5.6 TB/s), join 7.  Lookup of the same: 20, 4.6 TB/s.  With
// half of the tokens one id of a 32000 x 1024 table, 84 in all where 64 are taken
// without: the join of 512 tiles.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "columns.h"
#include "device_common.h"
#include "internal.h"

namespace dc {
namespace {

// ---------------------------------------------------------------------------
// Lookup: a wave takes kLookup tokens over 64 vectors of columns, their rows'
// loads in flight together.
// ---------------------------------------------------------------------------
constexpr int kLookup = 4;

template <class T, class Id>
__global__ void __launch_bounds__(256) k_lookup(int64_t T_, int64_t rows, int64_t D, const Id* ids, const T* table,
                                                int64_t ld_table, float scale, T* out, int64_t ld_out) {
  constexpr int V = 16 / sizeof(T);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * kLookup, j = ((int64_t)blockIdx.y * 64 + lane) * V;
  const int64_t left = D - j;
  if (left <= 0) return;
  float v[kLookup][V];
#pragma unroll
  for (int k = 0; k < kLookup; ++k) {
    const int64_t id = t0 + k < T_ ? (int64_t)ids[t0 + k] : -1;
    if (id >= 0 && id < rows) load_columns<T, V>(table + id * ld_table + j, left, v[k]);
    else
#pragma unroll
      for (int t = 0; t < V; ++t) v[k][t] = 0.f;
  }
#pragma unroll
  for (int k = 0; k < kLookup; ++k) {
    if (t0 + k >= T_) break;
#pragma unroll
    for (int t = 0; t < V; ++t) v[k][t] *= scale;
    store_columns<T, V>(out + (t0 + k) * ld_out + j, left, v[k]);
  }
}

// ---------------------------------------------------------------------------
// Sorting (id, token) by id: stable passes over `bits` bits of the id from the
// low ones up.  A workgroup of 1024 takes kSortTile tokens, each wave a run of
// them; a token's place is the number of tokens with smaller digits, plus
// those of its digit in earlier workgroups, earlier waves, and before it in
// its wave.  Ids outside the table sort behind it, as `rows`.
// ---------------------------------------------------------------------------
constexpr int kSortItems = 2;
constexpr int kSortTile = 1024 * kSortItems;
constexpr int kMostBits = 10;                 // of a pass
constexpr int kDigits = 1 << kMostBits;
// (Workgroups of 1024, 2048 and 4096 tokens: 32768 take 69, 68 and 73 us with
// all that follows.)
// Tiles up to which every workgroup adds the counts up by itself; for more a
// launch of its own does (that from 2 on, and 64 at once: 32768 tokens x 1024 68
// and 67 us where 16 take 64; 65536 x 1024 99 and 98, 16 99; 131072 x 512 103 and 98,
// 16 102).
constexpr int kSortSelf = 16;

template <class Id>
__device__ __forceinline__ uint32_t key_of(Id id, uint32_t rows) {
  return id >= 0 && (uint64_t)id < rows ? (uint32_t)id : rows;
}

struct SortPass {
  int64_t n;
  const uint32_t* keys;     // NULL: the ids themselves, token t at place t
  const uint32_t* tokens;
  uint32_t* out_keys;
  uint32_t* out_tokens;
  uint32_t* counts;         // [tiles + 1][kDigits]; the last row the totals, when scanned
  int32_t tiles, scanned;
  uint32_t rows;
  int32_t shift, bits;
};

template <class Id>
__device__ __forceinline__ uint32_t sort_key(const SortPass& p, const Id* ids, int64_t i) {
  return p.keys ? p.keys[i] : key_of(ids[i], p.rows);
}

// counts[tile][digit] of every tile.
template <class Id>
__global__ void __launch_bounds__(1024) k_sort_count(SortPass p, const Id* ids) {
  __shared__ uint32_t count[kDigits];
  const uint32_t mask = (1u << p.bits) - 1;
  count[threadIdx.x] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * kSortTile + threadIdx.x;
  uint32_t key[kSortItems];
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) key[k] = i0 + k * 1024 < p.n ? sort_key(p, ids, i0 + k * 1024) : 0;
#pragma unroll
  for (int k = 0; k < kSortItems; ++k)
    if (i0 + k * 1024 < p.n) atomicAdd(&count[(key[k] >> p.shift) & mask], 1u);
  __syncthreads();
  p.counts[(int64_t)blockIdx.x * kDigits + threadIdx.x] = count[threadIdx.x];
}

// Every digit's counts become the numbers of its tokens in earlier tiles; the
// totals go behind them.  A wave for 64 neighbouring digits, 16 tiles' loads
// in flight.
__global__ void __launch_bounds__(64) k_sort_scan(uint32_t* counts, int32_t tiles) {
  const int d = blockIdx.x * 64 + threadIdx.x;
  uint32_t sum = 0;
  for (int32_t b = 0; b < tiles; b += 16) {
    uint32_t c[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) c[k] = b + k < tiles ? counts[(int64_t)(b + k) * kDigits + d] : 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (b + k < tiles) counts[(int64_t)(b + k) * kDigits + d] = sum;
      sum += c[k];
    }
  }
  counts[(int64_t)tiles * kDigits + d] = sum;
}

// One pass over one tile.
template <class Id>
__device__ __forceinline__ void sort_pass(const SortPass& p, const Id* ids) {
  __shared__ uint32_t place[16][kDigits];  // counts, then first places, by wave
  __shared__ uint32_t wave_total[16];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, d = threadIdx.x;
  const uint32_t mask = (1u << p.bits) - 1;
  const int64_t i0 = (int64_t)blockIdx.x * kSortTile;
  uint32_t key[kSortItems], token[kSortItems], rank[kSortItems];
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int64_t i = i0 + (wave * kSortItems + k) * 64 + lane;
    key[k] = i < p.n ? sort_key(p, ids, i) : 0;
    token[k] = i < p.n ? (p.keys ? p.tokens[i] : (uint32_t)i) : 0;
  }
  // of this digit: tokens in earlier tiles, and in all (one tile: in its waves)
  uint32_t earlier = 0, total = 0;
  if (p.tiles > 1 && p.scanned) {
    earlier = p.counts[(int64_t)blockIdx.x * kDigits + d];
    total = p.counts[(int64_t)p.tiles * kDigits + d];
  } else if (p.tiles > 1) {
    for (int32_t b = 0; b < p.tiles; b += kSortSelf) {
      uint32_t c[kSortSelf];
#pragma unroll
      for (int k = 0; k < kSortSelf; ++k) c[k] = b + k < p.tiles ? p.counts[(int64_t)(b + k) * kDigits + d] : 0;
#pragma unroll
      for (int k = 0; k < kSortSelf; ++k) {
        earlier += b + k < (int32_t)blockIdx.x ? c[k] : 0;
        total += c[k];
      }
    }
  }
  if (d <= (int)mask)
#pragma unroll
    for (int w = 0; w < 16; ++w) place[w][d] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const bool in = i0 + (wave * kSortItems + k) * 64 + lane < p.n;
    const uint32_t g = (key[k] >> p.shift) & mask;
    uint64_t same = __ballot(in);
    for (int b = 0; b < p.bits; ++b) {
      const bool one = (g >> b) & 1;
      const uint64_t ones = __ballot(one);
      same &= one ? ones : ~ones;
    }
    const int before = __popcll(same & ((1ull << lane) - 1));
    uint32_t old = 0;
    if (in && before == 0) old = atomicAdd(&place[wave][g], (uint32_t)__popcll(same));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the next item's lanes see it
    old = __shfl(old, in ? __ffsll((unsigned long long)same) - 1 : lane);
    rank[k] = old + before;
  }
  __syncthreads();
  uint32_t mine[16];
#pragma unroll
  for (int w = 0; w < 16; ++w) mine[w] = d <= (int)mask ? place[w][d] : 0;
  if (p.tiles == 1)
#pragma unroll
    for (int w = 0; w < 16; ++w) total += mine[w];
  // the digit's first place: tokens of smaller digits, then of earlier tiles
  uint32_t first = total;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = __shfl_up(first, o);
    if (lane >= o) first += up;
  }
  if (lane == 63) wave_total[wave] = first;
  __syncthreads();
  uint32_t at = first - total + earlier;
#pragma unroll
  for (int w = 0; w < 16; ++w) at += w < wave ? wave_total[w] : 0;
  if (d <= (int)mask)
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      place[w][d] = at;
      at += mine[w];
    }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    if (i0 + (wave * kSortItems + k) * 64 + lane >= p.n) continue;
    const uint32_t to = place[wave][(key[k] >> p.shift) & mask] + rank[k];
    p.out_keys[to] = key[k];
    p.out_tokens[to] = token[k];
  }
}

template <class Id>
__global__ void __launch_bounds__(1024) k_sort_pass(SortPass p, const Id* ids) {
  sort_pass(p, ids);
}

// Every pass over a single tile, in one launch.
struct SortPasses {
  SortPass pass[3];
  int32_t count;
};
template <class Id>
__global__ void __launch_bounds__(1024) k_sort_tile(SortPasses s, const Id* ids) {
  for (int k = 0; k < s.count; ++k) {
    if (k) __syncthreads();  // the last pass is written, and its places are free
    sort_pass(s.pass[k], ids);
  }
}

// ---------------------------------------------------------------------------
// Sums of rows.
// ---------------------------------------------------------------------------
// Tiles that a workgroup of the join looks at (2 and 16: 32768 tokens x 1024 65 and 68
// us where 4 take 64; 1511 x 515 24 and 28, 4 24; half of the tokens one id 74 and
// 76, 4 84).
constexpr int kJoinTiles = 4;
// Rows of dE that a workgroup of the fill looks at (2 and 32: 32000 x 4096
// 132 and 135 us where 8 take 130).
constexpr int kFill = 8;

struct RowSums {
  int64_t n, rows, D;
  const uint32_t* keys;
  const uint32_t* tokens;
  const void* dy;
  int64_t ld_dy;
  void* dtable;
  int64_t ld;
  int32_t tile;    // sorted tokens per wave
  float* partial;  // [tiles][2][D]: of the row that came in from the tile before, of the one that goes on
  float scale;
  int32_t accumulate;
  uint32_t sum_blocks, across;  // workgroups that add up, across the columns
};

// The first place with a key of at least `key`.
__device__ __forceinline__ int64_t lower_bound(const uint32_t* keys, int64_t n, uint32_t key) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (keys[mid] < key) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// Rows that no token names become zeros: a workgroup looks at kFill of them,
// each lane at one, and writes whole rows.
template <class G>
__device__ __forceinline__ void fill_rows(const RowSums& a, int64_t block, int64_t blocks) {
  constexpr int V = 16 / sizeof(G);
  const int lane = threadIdx.x & 63;
  for (int64_t r0 = block * kFill; r0 < a.rows; r0 += blocks * kFill) {
    const int64_t r = r0 + lane;
    bool named = lane >= kFill || r >= a.rows;
    if (!named) {
      const int64_t at = lower_bound(a.keys, a.n, (uint32_t)r);
      named = at < a.n && a.keys[at] == (uint32_t)r;
    }
    uint64_t todo = ~__ballot(named);
    while (todo) {
      const int i = __ffsll((unsigned long long)todo) - 1;
      todo &= todo - 1;
      G* to = static_cast<G*>(a.dtable) + (r0 + i) * a.ld;
      for (int64_t j = (int64_t)threadIdx.x * V; j < a.D; j += 256 * V) {
        if (a.D - j >= V) {
          __builtin_nontemporal_store(u32x4_any{0, 0, 0, 0}, reinterpret_cast<u32x4_any*>(to + j));
        } else {
          for (int64_t k = j; k < a.D; ++k) to[k] = (G)0.f;
        }
      }
    }
  }
}

// The first workgroups add up the tiles' rows, the others write the zero rows
// beside them (32000 x 4096 fp32 from 8192 tokens: 101 us, 591 MB at 5.8 TB/s;
// in two launches 92 of zeros and 23 of rows).
template <class T, class G>
__global__ void __launch_bounds__(256) k_row_sums(RowSums a) {
  if (blockIdx.x >= a.sum_blocks) {
    fill_rows<G>(a, blockIdx.x - a.sum_blocks, gridDim.x - a.sum_blocks);
    return;
  }
  constexpr int V = 16 / sizeof(T);  // columns per lane
  constexpr int kAhead = 32 / V;     // rows in flight
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t j = ((int64_t)(blockIdx.x % a.across) * 64 + lane) * V, left = a.D - j;
  G* dtable = static_cast<G*>(a.dtable) + j;
  const int64_t tile = (int64_t)(blockIdx.x / a.across) * 4 + wave, p0 = tile * a.tile;
  // lanes past the last column stay: the tile's keys are held across the wave
  if (p0 >= a.n) return;
  const int have = a.n - p0 < a.tile ? (int)(a.n - p0) : a.tile;
  // lane i holds place p0 + i - 1: the tile, with the places before and after it
  const int64_t mine = p0 + lane - 1;
  const bool exists = lane <= have + 1 && mine >= 0 && mine < a.n;
  const uint32_t key = exists ? a.keys[mine] : (uint32_t)a.rows;
  const uint32_t token = exists ? a.tokens[mine] : 0;
  const uint32_t outside = (uint32_t)a.rows;
  auto key_at = [&](int i) { return (uint32_t)__builtin_amdgcn_readlane((int)key, i + 1); };
  const uint32_t first = key_at(0), last = key_at(have - 1);
  const bool came = p0 > 0 && key_at(-1) == first, goes = p0 + have < a.n && key_at(have) == last;
  const T* dy = static_cast<const T*>(a.dy) + j;
  float sum[V] = {};
  for (int i0 = 0; i0 < have; i0 += kAhead) {
    float v[kAhead][V], old[kAhead][V];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k;
      if (i >= have || key_at(i) == outside) break;
      load_columns<T, V>(dy + (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)token, i + 1) * a.ld_dy, left, v[k]);
      if (a.accumulate && key_at(i) != key_at(i + 1)) load_columns<G, V>(dtable + (int64_t)key_at(i) * a.ld, left, old[k]);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k;
      if (i >= have || key_at(i) == outside) break;
#pragma unroll
      for (int t = 0; t < V; ++t) sum[t] += v[k][t];
      const bool ends = i == have - 1 || key_at(i) != key_at(i + 1);
      if (!ends) continue;
      const bool in = came && key_at(i) == first, on = goes && i == have - 1;
      if (in || on) {
        store_columns<float, V>(a.partial + (tile * 2 + (in ? 0 : 1)) * a.D + j, left, sum);
      } else {
        float y[V];
#pragma unroll
        for (int t = 0; t < V; ++t) y[t] = a.scale * sum[t] + (a.accumulate ? old[k][t] : 0.f);
        store_columns<G, V>(dtable + (int64_t)key_at(i) * a.ld, left, y);
      }
#pragma unroll
      for (int t = 0; t < V; ++t) sum[t] = 0.f;
    }
  }
}

// A row whose tokens reach over tiles: the wave of the tile in which it ends
// adds up its partial sums, kJoin loads in flight; with more than a few of
// them the workgroup's four waves take a run each.  In fp64: a token of half a
// batch has thousands of parts, and in fp32 the error grew with their number.
constexpr int kJoin = 8;  // (4 and 16: 64 and 67 us where 8 take 64; 65536 tokens 101 and 104, 8 99)

template <class G>
__global__ void __launch_bounds__(256) k_row_join(RowSums a) {
  constexpr int V = 4;
  __shared__ double part[4][64][V];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t tiles = (a.n + a.tile - 1) / a.tile, base = (int64_t)blockIdx.x * kJoinTiles;
  // lane i looks at the tile base + i: whether a row that came in ends there
  const int64_t mine = base + lane, p0 = mine * a.tile, p1 = p0 + a.tile < a.n ? p0 + a.tile : a.n;
  uint32_t first = 0;
  bool ends = false;
  if (lane < kJoinTiles && mine > 0 && mine < tiles) {
    first = a.keys[p0];
    ends = first < a.rows && a.keys[p0 - 1] == first && (p1 == a.n || a.keys[p1] != first);
  }
  uint64_t todo = __ballot(ends);
  const int64_t j = ((int64_t)blockIdx.y * 64 + lane) * V, left = a.D - j;
  while (todo) {
    const int at = __ffsll((unsigned long long)todo) - 1;
    todo &= todo - 1;
    const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)first, at);
    const int64_t tile = base + at;
    // the tiles before it that the row came into, 64 at a time
    int64_t from = tile;
    for (;;) {
      const int64_t k = from - 1 - lane;
      const uint64_t came = __ballot(k > 0 && a.keys[k > 0 ? k * a.tile - 1 : 0] == key && a.keys[k > 0 ? k * a.tile : 0] == key);
      const int n = came == ~0ull ? 64 : __ffsll((unsigned long long)~came) - 1;
      from -= n;
      if (n < 64) break;
    }
    --from;  // the one that it begins in
    const int64_t parts = tile - from + 1;
    const bool alone = parts <= 2 * kJoin;
    if (alone && wave != (at & 3)) continue;
    const int64_t per = alone ? parts : (parts + 3) / 4, k0 = alone ? 0 : wave * per;
    const int64_t k1 = k0 + per < parts ? k0 + per : parts;
    G* to = static_cast<G*>(a.dtable) + (int64_t)key * a.ld + j;
    double sum[V] = {};
    float y[V] = {};
    if (a.accumulate && (alone || wave == 0)) load_columns<G, V>(to, left, y);
    for (int64_t k = k0; k < k1; k += kJoin) {
      float v[kJoin][V];
#pragma unroll
      for (int u = 0; u < kJoin; ++u)
        load_columns<float, V>(a.partial + ((from + k + u) * 2 + (k + u == 0 ? 1 : 0)) * a.D + j, k + u < k1 ? left : 0, v[u]);
#pragma unroll
      for (int u = 0; u < kJoin; ++u)
#pragma unroll
        for (int t = 0; t < V; ++t) sum[t] += v[u][t];
    }
    if (!alone) {
      __syncthreads();
#pragma unroll
      for (int t = 0; t < V; ++t) part[wave][lane][t] = sum[t];
      __syncthreads();
      if (wave) continue;
#pragma unroll
      for (int t = 0; t < V; ++t) sum[t] = (part[0][lane][t] + part[1][lane][t]) + (part[2][lane][t] + part[3][lane][t]);
    }
#pragma unroll
    for (int t = 0; t < V; ++t) y[t] = (float)((double)a.scale * sum[t] + (double)y[t]);
    store_columns<G, V>(to, left, y);
  }
}

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

// Where the workspace holds what: two buffers of keys and tokens, the counts,
// the partial sums.
struct EmbeddingSpace {
  int64_t sort_tiles, tile, tiles, keys_at[2], tokens_at[2], counts_at, partial_at, bytes;
  EmbeddingSpace(int32_t dtype, int64_t T, int64_t D) {
    sort_tiles = (T + kSortTile - 1) / kSortTile;
    // The longest tile that leaves eight waves a compute unit: long ones leave
    // fewer partial sums (32768 tokens x 1024: 32 64 us, 16 68), short ones finish
    // sooner (1511 x 515 fp32: 8 23 us, 16 27, 32 36).
    const int64_t per = 64 * (16 / (dtype == DC_F32 ? 4 : 2)), across = (D + per - 1) / per;
    for (tile = 32; tile > 8 && (T + tile - 1) / tile * across < 2048; tile /= 2) {
    }
    tiles = (T + tile - 1) / tile;
    int64_t at = 0;
    for (int k = 0; k < 2; ++k) {
      keys_at[k] = at;
      at += up16(4 * T);
      tokens_at[k] = at;
      at += up16(4 * T);
    }
    counts_at = at;
    if (sort_tiles > 1) at += (sort_tiles + 1) * kDigits * 4;
    partial_at = at;
    if (tiles > 1) at += up16(tiles * 2 * D * 4);
    bytes = at;
  }
};

template <class Id>
int sort_tokens(int64_t T, int64_t rows, const void* ids, char* ws, const EmbeddingSpace& e, hipStream_t stream) {
  int32_t bits = 1;
  while (rows >> bits) ++bits;  // keys are 0 .. rows
  const int32_t passes = (bits + kMostBits - 1) / kMostBits, each = (bits + passes - 1) / passes;
  const Id* id = static_cast<const Id*>(ids);
  SortPasses s{};
  s.count = passes;
  for (int32_t k = 0; k < passes; ++k) {
    SortPass& p = s.pass[k];
    p.n = T;
    if (k) {
      p.keys = reinterpret_cast<uint32_t*>(ws + e.keys_at[(k - 1) & 1]);
      p.tokens = reinterpret_cast<uint32_t*>(ws + e.tokens_at[(k - 1) & 1]);
    }
    p.out_keys = reinterpret_cast<uint32_t*>(ws + e.keys_at[k & 1]);
    p.out_tokens = reinterpret_cast<uint32_t*>(ws + e.tokens_at[k & 1]);
    p.tiles = (int32_t)e.sort_tiles;
    p.scanned = p.tiles > kSortSelf;
    p.rows = (uint32_t)rows;
    p.shift = k * each;
    p.bits = std::min(each, bits - p.shift);
    p.counts = reinterpret_cast<uint32_t*>(ws + e.counts_at);
    if (p.tiles == 1) continue;
    k_sort_count<Id><<<dim3((uint32_t)p.tiles), 1024, 0, stream>>>(p, id);
    if (p.scanned) k_sort_scan<<<kDigits / 64, 64, 0, stream>>>(p.counts, p.tiles);
    k_sort_pass<Id><<<dim3((uint32_t)p.tiles), 1024, 0, stream>>>(p, id);
  }
  if (e.sort_tiles == 1) k_sort_tile<Id><<<1, 1024, 0, stream>>>(s, id);
  return (passes - 1) & 1;
}

template <class T, class G>
void row_sums(const RowSums& s, int64_t tiles, hipStream_t stream) {
  RowSums a = s;
  constexpr int64_t per = 64 * (sizeof(T) == 2 ? 8 : 4);
  const uint32_t across = (uint32_t)((a.D + per - 1) / per);
  a.across = across;
  a.sum_blocks = (uint32_t)((tiles + 3) / 4) * across;
  const int64_t fill = a.accumulate ? 0 : std::min<int64_t>((a.rows + kFill - 1) / kFill, (int64_t)1 << 20);
  if (a.sum_blocks + fill) k_row_sums<T, G><<<dim3((uint32_t)(a.sum_blocks + fill)), 256, 0, stream>>>(a);
  if (tiles > 1)
    k_row_join<G><<<dim3((uint32_t)((tiles + kJoinTiles - 1) / kJoinTiles), (uint32_t)((a.D + 255) / 256)), 256, 0,
                    stream>>>(a);
}

}  // namespace

hipError_t launch_embedding(int32_t dtype, int32_t id_bytes, int64_t T, int64_t rows, int64_t D, const void* ids,
                            const void* table, int64_t ld_table, float scale, void* out, int64_t ld_out,
                            hipStream_t stream) {
  if (T == 0) return hipSuccess;
  auto launch = [&](auto type, auto id) {
    using E = decltype(type);
    using Id = decltype(id);
    constexpr int64_t per = 64 * (16 / sizeof(E));
    const dim3 grid((uint32_t)((T + 4 * kLookup - 1) / (4 * kLookup)), (uint32_t)((D + per - 1) / per));
    k_lookup<E, Id><<<grid, 256, 0, stream>>>(T, rows, D, static_cast<const Id*>(ids), static_cast<const E*>(table),
                                              ld_table, scale, static_cast<E*>(out), ld_out);
  };
  if (dtype == DC_BF16) id_bytes == 8 ? launch(__bf16{}, int64_t{}) : launch(__bf16{}, int32_t{});
  else id_bytes == 8 ? launch(float{}, int64_t{}) : launch(float{}, int32_t{});
  return hipGetLastError();
}

int64_t embedding_workspace(int32_t dtype, int64_t T, int64_t D) { return EmbeddingSpace(dtype, T, D).bytes; }

hipError_t launch_embedding_backward(int32_t dtype, int32_t grad_dtype, int32_t id_bytes, int64_t T, int64_t rows,
                                     int64_t D, const void* dy, int64_t ld_dy, const void* ids, float scale,
                                     void* dtable, int64_t ld, int32_t accumulate, void* workspace,
                                     hipStream_t stream) {
  if (T == 0 && accumulate) return hipSuccess;
  const EmbeddingSpace e(dtype, T, D);
  char* ws = static_cast<char*>(workspace);
  int at = 0;
  if (T) at = id_bytes == 8 ? sort_tokens<int64_t>(T, rows, ids, ws, e, stream)
                            : sort_tokens<int32_t>(T, rows, ids, ws, e, stream);
  RowSums a{};
  a.n = T;
  a.rows = rows;
  a.D = D;
  a.keys = reinterpret_cast<const uint32_t*>(ws + e.keys_at[at]);
  a.tokens = reinterpret_cast<const uint32_t*>(ws + e.tokens_at[at]);
  a.dy = dy;
  a.ld_dy = ld_dy;
  a.dtable = dtable;
  a.ld = ld;
  a.partial = reinterpret_cast<float*>(ws + e.partial_at);
  a.tile = (int32_t)e.tile;
  a.scale = scale;
  a.accumulate = accumulate;
  if (dtype == DC_F32) row_sums<float, float>(a, e.tiles, stream);
  else if (grad_dtype == DC_F32) row_sums<__bf16, float>(a, e.tiles, stream);
  else row_sums<__bf16, __bf16>(a, e.tiles, stream);
  return hipGetLastError();
}

}  // namespace dc
