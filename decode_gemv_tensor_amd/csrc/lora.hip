// Low-rank adapters beside a shared projection, forward and backward.
//
//   h[t] = A[i] x[t]              y[t] = base[t] + s[i] B[i] h[t]
//   g[t] = s[i] B[i]^T dy[t]      dx[t] = dx_base[t] + A[i]^T g[t]
//   dA[i] = sum_t g[t] x[t]^T     dB[i] = sum_t s[i] dy[t] h[t]^T
//
// for i = ids[t]. A rank is small beside n and k (4 R flop a value of base, dy
// or x, some 60 at rank 16 and 250 at 64, against a ridge of 200 and more), so
// memory bounds all of it, and launches where rows are few. The forward is two
// kernels (h; y), or one for the fewest rows; the backward sorts the rows, then
// g, dx and the gradients. Every product runs on bf16 MFMA in fp32, with h and
// g, which are fp32, as three bf16 terms.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "binade.h"
#include "device_common.h"

namespace binade {
namespace {

using namespace dev;

struct LoraArgs {
  const uint16_t *a, *b;
  const float* scale;
  const int32_t* ids;
  int64_t n, k, m;
  int32_t rank, n_adapters;
  uint32_t* status;
};

__device__ __forceinline__ float bf16_f32(uint16_t v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

__device__ __forceinline__ int32_t adapter_of(const LoraArgs& p, int64_t t) {
  const int32_t i = p.ids != nullptr ? p.ids[t] : 0;
  return i >= 0 && i < p.n_adapters ? i : -1;
}

__device__ __forceinline__ float load_any(const void* v, int64_t i, bool is_bf16) {
  return is_bf16 ? bf16_f32(static_cast<const uint16_t*>(v)[i])
                 : static_cast<const float*>(v)[i];
}

__device__ __forceinline__ void store_any(void* v, int64_t i, bool is_bf16, float f) {
  if (is_bf16)
    static_cast<uint16_t*>(v)[i] = to_bf16_rne(f);
  else
    static_cast<float*>(v)[i] = f;
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kRowTile = 32;   // rows sorted by adapter: of a tile
constexpr int kSlice = 256;    // columns whose products one MFMA chain adds
constexpr int kStreams = 8;    // running sums the slices are dealt to

__device__ __forceinline__ bf16x8 as_bf16x8(uint4 v) { return __builtin_bit_cast(bf16x8, v); }

// 16 bytes at any 2-byte alignment (rows of an odd length).
__device__ __forceinline__ uint4 load8(const uint16_t* p) {
  uint4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// The same of which only left elements exist; zeros for the others.
__device__ __forceinline__ uint4 load8_part(const uint16_t* p, int64_t left) {
  if (left >= 8) return load8(p);
  uint16_t v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < left ? p[j] : static_cast<uint16_t>(0);
  return __builtin_bit_cast(uint4, v);
}

// v = hi + mid + lo exactly, each a bf16 (8 significant bits by truncation):
// fp32 values enter a bf16 MFMA as three terms and lose nothing. Infinity
// and NaN stay in hi alone; an infinite value on the other side meets terms
// that are 0, see redo_nan.
__device__ __forceinline__ void split3(float v, uint16_t& hi, uint16_t& mid, uint16_t& lo) {
  const uint32_t u = __float_as_uint(v), top = u & 0xFFFF0000u;
  float rest = v - __uint_as_float(top);
  if ((u & 0x7F800000u) == 0x7F800000u) rest = 0.0f;
  const uint32_t m = __float_as_uint(rest) & 0xFFFF0000u;
  hi = static_cast<uint16_t>(top >> 16);
  mid = static_cast<uint16_t>(m >> 16);
  lo = static_cast<uint16_t>(__float_as_uint(rest - __uint_as_float(m)) >> 16);
}

// Blocks are dealt to the 8 XCDs round robin. This gives every XCD one run of
// consecutive units of work, so that neighbours, which read the same
// adapter, meet in one L2. Launched over xcd_grid(units) blocks; a unit of
// units or more has no work.
constexpr int64_t kXcds = 8;
__device__ __forceinline__ int64_t xcd_unit() {
  return static_cast<int64_t>(blockIdx.x % kXcds) * (gridDim.x / kXcds) + blockIdx.x / kXcds;
}
dim3 xcd_grid(int64_t units) {
  return dim3(static_cast<uint32_t>((units + kXcds - 1) / kXcds * kXcds));
}

// ---------------------------------------------------------------- forward
// h[t] = A[i] x[t]. Order, fixed by k alone: columns are cut into slices of
// 256; slice s is one MFMA chain c_s from +0.0 (step j: lane group g carries
// columns 256 s + 32 j + 8 g .. + 7); running sum w of 8 adds c_w, c_w+8, ...
// from +0.0; h adds the running sums in order from +0.0. MFMA rows are
// independent, so a row's bits do not depend on the rows beside it; a tile of
// 16 rows runs once for each adapter among them and every row keeps its own
// adapter's sum. The same order at three grains:
//  - whole: a block per tile, wave w = running sum w, joined through LDS;
//  - streams: a block per tile and running sum;
//  - slices: a block per tile and slice, for the fewest rows.
// The two finer ones deal the tile's adapters to the block's waves and leave
// partial sums [parts][m][rank] that the second product's kernel adds.
// The whole grain also splits h into the second product's MFMA operands.
// Measured: 4096 rows of 3840 columns, rank 64, 16 adapters, 23.7 us (x alone
// 6: A is read once a tile, 126 MB out of the L2, and a wave has its own
// loads' latency to wait for eight times); 61 rows of 15360, 32 adapters of
// rank 32, in slices 10.6 (A's 31 MB alone 6). Loading a slice ahead changed
// nothing, 101.0 and 101.1 us for both products of the 4096 rows.
//
// MFMA wants 16 rows in consecutive lanes, and a load whose neighbouring lanes
// sit in different rows costs the L1 one access a lane (64 of 16 bytes; that
// bound the first version). So every operand is loaded with four lanes on 64
// contiguous bytes of a row and turned round through 1 KB of LDS.
struct ShrinkArgs {
  LoraArgs p;              // a: [rank][k] per adapter, zeros from cols to k
  const uint16_t* x;
  float* out;              // streams, slices: partial sums [parts][m][rank]
  float* h;                // whole: fp32 [m][rank] or NULL
  uint4* frag;             // whole: [tiles][3][KS][64] operands (NULL otherwise)
  int64_t ldx, cols;       // columns of x
  int32_t slices, parts;   // parts: 1 (whole), 8 (streams) or slices
  // Rows sorted by adapter (Order below; kAny only) or NULL: then no tile is
  // mixed. tiles: of 16, at most.
  const int32_t *perm, *adapter, *tile0;
  int64_t tiles;
};

// A barrier that waits for LDS alone (__syncthreads() would also wait for the
// loads on their way).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// N operands as loaded (lane 4 row + octet) -> as MFMA takes them (lane row +
// 16 octet), through N KB of the wave's own; the swizzle spreads the reads of
// 8 lanes over all banks.
template <int N>
__device__ __forceinline__ void turn(uint4 (&v)[N], uint4* lds, int lane) {
#pragma unroll
  for (int j = 0; j < N; ++j) lds[64 * j + (lane ^ ((lane >> 4) & 3))] = v[j];
  wave_sync();
  const int i = lane & 15, g = lane >> 4;
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = lds[64 * j + 4 * i + (g ^ ((i >> 2) & 3))];
  wave_sync();
}

// The sums of a tile of 16 rows over slices first, first + step, ...: lane
// (i, g) gets rank 16 r + i of rows 4 g + q in mine[r][q] (zeros without
// adapter). With deal > 0 the tile's adapters are dealt to that many waves;
// the result's bits say which rows this wave holds. id: of the tile's row i, -1
// behind the last; lrow: the row a lane loads, the tile's row lane / 4 (any
// one in place of one that does not exist). kAny: rows of x at any 2-byte alignment and of any length
// (gradients of an odd number of outputs); otherwise 16-byte aligned, a
// multiple of 32.
template <int RT, bool kAny>
__device__ __forceinline__ uint32_t shrink_rows(const ShrinkArgs& s, int64_t lrow, int32_t id,
                                                int32_t first, int32_t step, int32_t deal,
                                                int wave, int lane, uint4* stage,
                                                floatx4 (&mine)[RT]) {
  const LoraArgs& p = s.p;
  const int i = lane & 15, g = lane >> 4;
  int32_t idq[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) idq[q] = __shfl(id, 4 * g + q, 64);
#pragma unroll
  for (int r = 0; r < RT; ++r) mine[r] = floatx4{0, 0, 0, 0};
  const uint16_t* xl = s.x + lrow * s.ldx + 8 * (lane & 3);
  uint32_t todo = static_cast<uint32_t>(__ballot(id >= 0)) & 0xFFFFu;
  uint32_t got = wave == 0 ? 0xFFFFu & ~todo : 0u;
  for (int32_t nth = 0; todo != 0; ++nth) {
    const int32_t a = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    const uint32_t match = static_cast<uint32_t>(__ballot(id == a)) & 0xFFFFu;
    todo &= ~match;
    if (deal > 0 && nth % deal != wave) continue;
    got |= match;
    const uint16_t* aa = p.a + static_cast<int64_t>(a) * p.rank * p.k;
    const auto rank_row = [&](int r) { return r < p.rank ? r : p.rank - 1; };
    floatx4 sum[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) sum[r] = floatx4{0, 0, 0, 0};
    uint4 xf[8], af[8];
    const auto load_x = [&](int32_t c, auto part) __attribute__((always_inline)) {
      const int64_t col = static_cast<int64_t>(c) * kSlice;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint16_t* from = xl + col + 32 * j;
        const int64_t left = s.cols - col - 32 * j;
        if (!part || left >= 32) {
          xf[j] = kAny ? load8(from) : *reinterpret_cast<const uint4*>(from);
        } else {
          xf[j] = uint4{0, 0, 0, 0};
          if (kAny && left > 0) xf[j] = load8_part(from, left - 8 * (lane & 3));
        }
      }
    };
    const auto load_a = [&](int32_t c, auto part, int r) __attribute__((always_inline)) {
      const int64_t col = static_cast<int64_t>(c) * kSlice;
      const uint16_t* al = aa + rank_row(16 * r + (lane >> 2)) * p.k + 8 * (lane & 3) + col;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!part || s.cols - col > 32 * j)
          af[j] = *reinterpret_cast<const uint4*>(al + 32 * j);
        else
          af[j] = uint4{0, 0, 0, 0};
      }
    };
    // part: a last slice of fewer columns, zeros behind them
    const auto slice = [&](int32_t c, auto part) __attribute__((always_inline)) {
      floatx4 acc[RT];
      load_x(c, part);
      load_a(c, part, 0);
      turn(xf, stage, lane);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        acc[r] = floatx4{0, 0, 0, 0};
        uint4 bf[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) bf[j] = af[j];
        if (RT < 8 && r + 1 < RT) load_a(c, part, r + 1);   // 8 tiles' sums leave no registers
        turn(bf, stage, lane);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(xf[j]), as_bf16x8(bf[j]),
                                                           acc[r], 0, 0, 0);
        if (RT == 8 && r + 1 < RT) load_a(c, part, r + 1);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) sum[r] += acc[r];
    };
    const int32_t whole = static_cast<int32_t>(s.cols / kSlice);
    int32_t c = first;
#pragma unroll 1
    for (; c < whole; c += step) slice(c, std::false_type());
    if (c < s.slices) slice(c, std::true_type());
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (idq[q] == a) mine[r][q] = sum[r][q];
  }
  return got;
}

template <int RT, bool kAny>
__global__ __launch_bounds__(512) void shrink_kernel(ShrinkArgs s) {
  const LoraArgs& p = s.p;
  constexpr int kSumLd = 16 * RT + 4;
  __shared__ union {
    uint4 stage[kStreams][512];
    float sums[kStreams][16][kSumLd];
  } lds;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  // units: slice (or running sum) major, tiles of 16 rows minor
  const int64_t tiles = s.tiles, unit = xcd_unit();
  if (unit >= tiles * s.parts) return;
  const int32_t part = static_cast<int32_t>(unit / tiles);
  const int64_t tile = unit - part * tiles, row0 = tile * 16;
  int64_t row = row0 + i < p.m ? row0 + i : p.m - 1;
  int32_t id = row0 + i < p.m ? adapter_of(p, row) : -1;
  if (part == 0 && threadIdx.x < 16 && p.status != nullptr && p.ids != nullptr && id < 0 &&
      row0 + i < p.m && p.ids[row] != -1)
    atomicOr(p.status, static_cast<uint32_t>(BINADE_DEV_BAD_INDEX));
  bool exists = row0 + i < p.m;
  if (kAny && s.perm != nullptr) {
    if (row0 >= static_cast<int64_t>(s.tile0[p.n_adapters]) * kRowTile) return;
    const int32_t at = s.perm[row0 + i];
    exists = at >= 0;
    row = exists ? at : 0;
    id = exists ? s.adapter[row0 / kRowTile] : -1;
  }
  // of the row a lane loads
  const int32_t row32 = static_cast<int32_t>(row);
  const int64_t lrow = __shfl(row32, lane >> 2, 64);
  const bool whole = s.frag != nullptr;
  const int32_t first = whole ? wave : part;
  const int32_t step = whole || s.parts < s.slices ? kStreams : s.slices;
  floatx4 mine[RT];
  const uint32_t got =
      shrink_rows<RT, kAny>(s, lrow, id, first, step, whole ? 0 : blockDim.x >> 6, wave, lane,
                            lds.stage[wave], mine);
  if (!whole) {
    float* out = s.out + part * p.m * p.rank;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int32_t t = __shfl(exists ? row32 : -1, 4 * g + q, 64);
      if (t < 0 || !((got >> (4 * g + q)) & 1u)) continue;
#pragma unroll
      for (int r = 0; r < RT; ++r)
        if (16 * r + i < p.rank) out[static_cast<int64_t>(t) * p.rank + 16 * r + i] = mine[r][q];
    }
    return;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int q = 0; q < 4; ++q) lds.sums[wave][4 * g + q][16 * r + i] = mine[r][q];
  __syncthreads();
  // thread = (K step, lane) of the second product's operand: 8 ranks of a row
  const int32_t ks = (p.rank + 31) / 32;
  if (wave >= ks) return;
  const int32_t r0 = 32 * wave + 8 * g;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  if (kAny && s.perm != nullptr && !exists) return;
  const int64_t place = kAny && s.perm != nullptr ? row : row0 + i;
  if (r0 < p.rank && exists) {
    const int32_t live = s.slices < kStreams ? s.slices : kStreams;
    for (int32_t w = 0; w < live; ++w)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += lds.sums[w][i][r0 + j];
    if (s.h != nullptr) __builtin_memcpy(s.h + row * p.rank + r0, v, 32);
  }
  uint16_t d[3][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) split3(v[j], d[0][j], d[1][j], d[2][j]);
#pragma unroll
  for (int t = 0; t < 3; ++t)
    s.frag[((place / 16 * 3 + t) * ks + wave) * 64 + 16 * g + place % 16] =
        __builtin_bit_cast(uint4, d[t]);
}

// y[t] = base[t] + s[i] B[i] h[t]. Column c of a wave's MFMA tiles is spread so
// that lane i ends with the CT adjacent columns CT i .. CT i + CT - 1. A tile of
// 16 rows runs once for each adapter among them and every row keeps its own;
// base + scale * product is one fma (rows without an adapter: -0 * 0 + base).
// Two shapes, at 4096 rows of bf16 base and y, 15360 columns, rank 64, 75.5 us
// (252 MB, 3.3 TB/s; reading base and writing y alone 44: a wave's tile of 2 KB
// waits for its operands, and more waves have no registers) and at 61 rows of
// 3840 columns, fp32 base, 32 adapters of rank 32, 11.1:
//  - few rows: a block of four waves has 16 rows by 128 columns, joins the
//    partial sums of h in LDS and splits them into three bf16 terms there;
//  - many rows: a wave has 64 columns of eight row tiles; h arrives split as
//    operands, B's rows stay in the wave's LDS while the adapter does not
//    change (in registers they cost the occupancy that hides a tile's loads),
//    a tile's base is loaded while the one before it runs.
struct ExpandArgs {
  LoraArgs p;
  const float* part;       // few rows: partial sums of h
  const uint4* frag;       // many rows: h as operands
  const void* base;
  void* y;
  float* h;
  int64_t ld_base, ldy;
  int32_t parts;           // of the first product: 1, 8 or its slices
  int32_t base_kind;       // 0 none, 1 fp32, 2 bf16
  bool y_bf16;
  int32_t tiles;           // many rows: row tiles of a block
};

// The sum of a value's partial sums in the order of the first product, four
// ranks at a time, by two neighbouring lanes: the even one adds the running
// sums 0 to 3, the odd one goes on with 4 to 7 and has the result. at: the
// first of parts partials, next apart.
__device__ __forceinline__ floatx4 join_parts(const float* at, int64_t next, int32_t parts,
                                              int half) {
  constexpr int kAhead = 4, kHalf = kStreams / 2;
  floatx4 sum[kHalf];
#pragma unroll
  for (int w = 0; w < kHalf; ++w) sum[w] = floatx4{0, 0, 0, 0};
  for (int32_t c = kHalf * half; c < parts; c += kAhead * kStreams) {
    floatx4 d[kAhead][kHalf];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int w = 0; w < kHalf; ++w) {
        const int32_t q = c + j * kStreams + w;
        d[j][w] = floatx4{0, 0, 0, 0};
        if (q < parts) d[j][w] = *reinterpret_cast<const floatx4*>(at + q * next);
      }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int w = 0; w < kHalf; ++w) sum[w] += d[j][w];
  }
  floatx4 v{0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < kHalf; ++w) v += sum[w];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float o = __shfl_xor(v[r], 1, 64);
#pragma unroll
    for (int w = 0; w < kHalf; ++w) o += sum[w][r];
    v[r] = o;
  }
  return v;
}

// Kinds of base and y.
constexpr int kNone = 0, kF32 = 1, kBf16 = 2;

template <int CT, int BK>
struct BaseTile {
  uint32_t d[4][BK == kNone ? 1 : BK == kBf16 ? CT / 2 : CT];   // four rows' values, as loaded
};

// Where a lane's values of a tile lie: a uniform address per row q and one
// 32-bit byte offset for all of them (rows 4 g + q, columns col on).
template <int K>
__device__ __forceinline__ uint32_t lane_offset(int64_t ld, int g, int32_t col_in_wave) {
  return static_cast<uint32_t>(4 * g * ld + col_in_wave) * (K == kBf16 ? 2u : 4u);
}

template <int CT, int BK>
__device__ __forceinline__ void load_base(const ExpandArgs& s, int64_t row0, int32_t rows, int g,
                                          int64_t wave_col, int32_t col_in_wave, bool full,
                                          BaseTile<CT, BK>& to) {
  if (BK == kNone || !full) return;
  constexpr int kSize = BK == kBf16 ? 2 : 4;
  const char* at = static_cast<const char*>(s.base) + (row0 * s.ld_base + wave_col) * kSize;
  const uint32_t off = lane_offset<BK>(s.ld_base, g, col_in_wave);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (rows == 16 || 4 * g + q < rows)
      __builtin_memcpy(to.d[q], at + q * s.ld_base * kSize + off, CT * kSize);
}

// The same without a branch (a load under a condition is one that the compiler
// cannot count, and it waits for all loads instead of the oldest ones): rows
// behind the last are the last, the columns of a lane that is not full the
// row's last CT; neither is used. n >= CT.
template <int CT, int BK>
__device__ __forceinline__ void load_base_any(const ExpandArgs& s, int64_t row0, int32_t rows, int g,
                                              int64_t col, BaseTile<CT, BK>& to) {
  if (BK == kNone) return;
  constexpr uint32_t kSize = BK == kBf16 ? 2 : 4;
  const char* at = static_cast<const char*>(s.base) + row0 * s.ld_base * kSize;
  const uint32_t row_bytes = static_cast<uint32_t>(s.ld_base) * kSize;
  const uint32_t col_bytes = static_cast<uint32_t>(col) * kSize;
  uint32_t off[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) off[q] = 4 * g * row_bytes + col_bytes + q * row_bytes;
  if (rows < 16) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      off[q] = static_cast<uint32_t>(4 * g + q < rows ? 4 * g + q : rows - 1) * row_bytes + col_bytes;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) __builtin_memcpy(to.d[q], at + off[q], CT * kSize);
}

// Four rows' results from column col on: base + scale * product, stored.
template <int CT, int BK, int YK>
__device__ __forceinline__ void finish_rows(const ExpandArgs& s, int64_t row0, int32_t rows, int g,
                                            int64_t wave_col, int32_t col_in_wave, bool full,
                                            const BaseTile<CT, BK>& base,
                                            const floatx4 (&acc)[CT], const float (&scale)[4]) {
  constexpr int kSize = YK == kBf16 ? 2 : 4;
  if (full) {
    char* at = static_cast<char*>(s.y) + (row0 * s.ldy + wave_col) * kSize;
    const uint32_t off = lane_offset<YK>(s.ldy, g, col_in_wave);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float f[CT];
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        float b = 0.0f;
        if (BK == kBf16)
          b = c & 1 ? bf16_hi(base.d[q][c / 2]) : bf16_lo(base.d[q][c / 2]);
        else if (BK == kF32)
          b = __uint_as_float(base.d[q][c]);
        f[c] = __builtin_fmaf(scale[q], acc[c][q], b);
      }
      if (rows < 16 && 4 * g + q >= rows) continue;
      if (YK == kBf16) {
        uint32_t d[CT / 2];
#pragma unroll
        for (int c = 0; c < CT / 2; ++c) d[c] = pack_bf16(f[2 * c], f[2 * c + 1]);
        __builtin_memcpy(at + q * s.ldy * kSize + off, d, 2 * CT);
      } else {
        __builtin_memcpy(at + q * s.ldy * kSize + off, f, 4 * CT);
      }
    }
  } else if (wave_col + col_in_wave < s.p.n) {   // the row's last columns, one by one
    const int64_t col = wave_col + col_in_wave;
#pragma unroll
    for (int c = 0; c < CT - 1; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (4 * g + q >= rows || col + c >= s.p.n) continue;
        const int64_t t = row0 + 4 * g + q;
        const float b =
            BK == kNone ? 0.0f : load_any(s.base, t * s.ld_base + col + c, BK == kBf16);
        store_any(s.y, t * s.ldy + col + c, YK == kBf16, __builtin_fmaf(scale[q], acc[c][q], b));
      }
  }
}

__device__ __forceinline__ bool is_nan(float v) { return v != v; }

// Whether a lane has a NaN in v: two values a comparison.
template <int N>
__device__ __forceinline__ bool any_nan(const floatx4 (&v)[N]) {
  bool any = false;
#pragma unroll
  for (int c = 0; c < N; ++c)
    any |= __builtin_isunordered(v[c][0], v[c][1]) | __builtin_isunordered(v[c][2], v[c][3]);
  return any;
}

// An infinite value of B beside an h that fewer than three bf16 terms hold: the
// terms that are 0 make NaN of what is infinite. (The terms of a value have one
// sign, so nothing else goes wrong.) A NaN is formed again from h itself, rank
// by rank in fp32, and stays one if it is. h: (row of the tile, rank) -> h. id:
// of the tile's row in a lane.
template <int CT, typename H>
__device__ __forceinline__ void redo_nan(const LoraArgs& p, int32_t id, int64_t wave_col, int lane,
                                         floatx4 (&mine)[CT], H h) {
  if (__ballot(any_nan(mine)) == 0) return;
  asm volatile("" : "+v"(lane));   // nothing of this is kept through the caller's loop
  const int g = lane >> 4;
  const int64_t col = wave_col + CT * (lane & 15);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int32_t a = __shfl(id, 4 * g + q, 64);
    bool open = false;
#pragma unroll
    for (int c = 0; c < CT; ++c) open |= is_nan(mine[c][q]);
    if (a < 0 || col >= p.n || !open) continue;
    float sum[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) sum[c] = 0.0f;
#pragma unroll 1
    for (int32_t r = 0; r < p.rank && open; ++r) {
      const float v = h(4 * g + q, r);
      open = false;
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const int64_t n = col + c < p.n ? col + c : p.n - 1;
        sum[c] = __builtin_fmaf(v, bf16_f32(p.b[(a * p.n + n) * p.rank + r]), sum[c]);
        open |= !is_nan(sum[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) mine[c][q] = is_nan(mine[c][q]) ? sum[c] : mine[c][q];
  }
}

// B's operands of adapter a for a wave's columns, as loaded; turn() follows.
// Zeros for ranks beyond the last (h has zeros there too).
template <int KS, int CT>
__device__ __forceinline__ void load_b(const LoraArgs& p, int32_t a, int64_t wave_col, int lane,
                                       uint4 (&bf)[KS][CT]) {
  const uint16_t* b = p.b + static_cast<int64_t>(a) * p.n * p.rank;
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int64_t n = wave_col + CT * (lane >> 2) + c;
    const uint16_t* row = b + (n < p.n ? n : p.n - 1) * p.rank;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int32_t o = 32 * k + 8 * (lane & 3);
      bf[k][c] = *reinterpret_cast<const uint4*>(row + (o < p.rank ? o : 0));
    }
  }
  if (32 * KS > p.rank) {
    const bool live = 32 * (KS - 1) + 8 * (lane & 3) < p.rank;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      uint4& v = bf[KS - 1][c];
      v.x = live ? v.x : 0u;
      v.y = live ? v.y : 0u;
      v.z = live ? v.z : 0u;
      v.w = live ? v.w : 0u;
    }
  }
}

// A few-rows wave's products: 16 rows, h split in LDS, up to kBatch adapters'
// operands at once, so that a mixed tile waits for memory once per batch. The
// first batch is requested by begin(), ahead of h.
template <int KS, int CT>
struct FewRows {
  static constexpr int kBatch = KS <= 2 ? 4 : 2;
  int32_t a[kBatch];
  uint4 bf[kBatch][KS][CT];
  uint64_t todo;

  __device__ __forceinline__ void request(const LoraArgs& p, int32_t id, int64_t wave_col,
                                          int lane) {
#pragma unroll
    for (int z = 0; z < kBatch; ++z) {
      a[z] = todo != 0 ? __builtin_amdgcn_readlane(id, __builtin_ctzll(todo)) : a[0];
      todo &= ~__ballot(id == a[z]);
    }
#pragma unroll
    for (int z = 0; z < kBatch; ++z)
      if (z == 0 || a[z] != a[0]) load_b<KS, CT>(p, a[z], wave_col, lane, bf[z]);
  }

  __device__ __forceinline__ void begin(const LoraArgs& p, int32_t id, int64_t wave_col, int lane) {
    todo = __ballot(id >= 0) & 0xFFFFu;
    a[0] = -1;
    if (todo != 0) request(p, id, wave_col, lane);
  }

  __device__ __forceinline__ void multiply(const LoraArgs& p, int32_t id, int64_t wave_col,
                                           int lane, uint4* stage,
                                           const uint16_t (&hs)[3][16][32 * KS + 8],
                                           floatx4 (&mine)[CT], float (&scale)[4]) {
    const int i = lane & 15, g = lane >> 4;
    int32_t idq[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) idq[q] = __shfl(id, 4 * g + q, 64), scale[q] = -0.0f;
#pragma unroll
    for (int c = 0; c < CT; ++c) mine[c] = floatx4{0, 0, 0, 0};
    while (a[0] >= 0) {
#pragma unroll
      for (int z = 0; z < kBatch; ++z) {
        if (z > 0 && a[z] == a[0]) break;
#pragma unroll
        for (int k = 0; k < KS; ++k) turn(bf[z][k], stage, lane);
        const float sc = p.scale != nullptr ? p.scale[a[z]] : 1.0f;
        floatx4 acc[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[c] = floatx4{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int t3 = 0; t3 < 3; ++t3) {
            const bf16x8 hf =
                as_bf16x8(*reinterpret_cast<const uint4*>(&hs[t3][i][32 * k + 8 * g]));
#pragma unroll
            for (int c = 0; c < CT; ++c)
              acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hf, as_bf16x8(bf[z][k][c]), acc[c],
                                                               0, 0, 0);
          }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bool hit = idq[q] == a[z];
          scale[q] = hit ? sc : scale[q];
#pragma unroll
          for (int c = 0; c < CT; ++c) mine[c][q] = hit ? acc[c][q] : mine[c][q];
        }
      }
      if (todo == 0) break;
      request(p, id, wave_col, lane);
    }
    redo_nan(p, id, wave_col, lane, mine, [&](int t, int32_t r) {
      return (bf16_f32(hs[0][t][r]) + bf16_f32(hs[1][t][r])) + bf16_f32(hs[2][t][r]);
    });
  }
};

template <int KS, int BK, int YK>
__global__ __launch_bounds__(256) void expand_few_kernel(ExpandArgs s) {
  const LoraArgs& p = s.p;
  constexpr int CT = 2, kLd = 32 * KS + 8;
  __shared__ __align__(16) uint16_t hs[3][16][kLd];
  __shared__ uint4 stage[4][64 * CT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  // units: row tiles major, columns minor
  const int64_t col_blocks = (p.n + 64 * CT - 1) / (64 * CT), unit = xcd_unit();
  const int64_t row0 = unit / col_blocks * 16, col_block = unit % col_blocks;
  if (row0 >= p.m) return;
  const int32_t rows = static_cast<int32_t>(p.m - row0 < 16 ? p.m - row0 : 16);
  const int64_t wave_col = (col_block * 4 + uniform(wave)) * (16 * CT);
  const bool full = wave_col + CT * i + CT <= p.n;
  const int32_t id = i < rows ? adapter_of(p, row0 + i) : -1;
  BaseTile<CT, BK> base;
  load_base<CT, BK>(s, row0, rows, g, wave_col, CT * i, full, base);
  FewRows<KS, CT> tile;
  tile.begin(p, id, wave_col, lane);
  for (int32_t e = threadIdx.x; e < 2 * 16 * 8 * KS; e += 256) {
    const int32_t half = e & 1, t = e / (16 * KS), r = 4 * (e / 2 % (8 * KS));
    floatx4 v{0, 0, 0, 0};
    if (r < p.rank && t < rows) {
      const int64_t at = (row0 + t) * p.rank + r;
      v = join_parts(s.part + at, p.m * p.rank, s.parts, half);
      if (half && s.h != nullptr && col_block == 0) *reinterpret_cast<floatx4*>(s.h + at) = v;
    }
    if (!half) continue;
    uint16_t d[3][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) split3(v[j], d[0][j], d[1][j], d[2][j]);
#pragma unroll
    for (int t3 = 0; t3 < 3; ++t3) __builtin_memcpy(&hs[t3][t][r], d[t3], 8);
  }
  __syncthreads();
  floatx4 mine[CT];
  float scale[4];
  tile.multiply(p, id, wave_col, lane, stage[wave], hs, mine, scale);
  finish_rows<CT, BK, YK>(s, row0, rows, g, wave_col, CT * i, full, base, mine, scale);
}

// The fewest rows in one launch: a block of eight waves (16 rows by 256
// columns) forms h of its rows anew, in the whole grain's order, while B and
// base are on their way. Reading A once a block costs less than a second
// launch while A's rows for the tile stay small.
template <int RT, int BK, int YK>
__global__ __launch_bounds__(512) void one_pass_kernel(ShrinkArgs sh, ExpandArgs s) {
  constexpr int CT = 2, KS = (RT + 1) / 2, kLd = 32 * KS + 8, kSumLd = 16 * RT + 4;
  const LoraArgs& p = s.p;
  __shared__ union {
    uint4 stage[kStreams][512];
    float sums[kStreams][16][kSumLd];
  } lds;
  __shared__ __align__(16) uint16_t hs[3][16][kLd];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), i = lane & 15, g = lane >> 4;
  const int32_t rows = static_cast<int32_t>(p.m);
  const int64_t wave_col = (static_cast<int64_t>(blockIdx.x) * 8 + wave) * (16 * CT);
  const bool full = wave_col + CT * i + CT <= p.n;
  const int32_t id = i < rows ? adapter_of(p, i) : -1;
  if (blockIdx.x == 0 && threadIdx.x < 16 && p.status != nullptr && p.ids != nullptr && id < 0 &&
      i < rows && p.ids[i] != -1)
    atomicOr(p.status, static_cast<uint32_t>(BINADE_DEV_BAD_INDEX));
  BaseTile<CT, BK> base;
  load_base<CT, BK>(s, 0, rows, g, wave_col, CT * i, full, base);
  FewRows<KS, CT> tile;
  tile.begin(p, id, wave_col, lane);
  floatx4 part[RT];
  shrink_rows<RT, false>(sh, (lane >> 2) < rows ? lane >> 2 : rows - 1, id, wave, kStreams, 0, wave,
                         lane, lds.stage[wave], part);
  __syncthreads();
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int q = 0; q < 4; ++q) lds.sums[wave][4 * g + q][16 * r + i] = part[r][q];
  __syncthreads();
  const int32_t live = sh.slices < kStreams ? sh.slices : kStreams;
  for (int32_t e = threadIdx.x; e < 16 * 32 * KS; e += 512) {
    const int32_t t = e / (32 * KS), r = e % (32 * KS);
    float v = 0.0f;
    if (r < p.rank && t < rows) {
      for (int32_t w = 0; w < live; ++w) v += lds.sums[w][t][r];
      if (s.h != nullptr && blockIdx.x == 0) s.h[t * p.rank + r] = v;
    }
    split3(v, hs[0][t][r], hs[1][t][r], hs[2][t][r]);
  }
  __syncthreads();
  if (wave_col >= p.n) return;
  floatx4 mine[CT];
  float scale[4];
  tile.multiply(p, id, wave_col, lane, lds.stage[wave], hs, mine, scale);
  finish_rows<CT, BK, YK>(s, 0, rows, g, wave_col, CT * i, full, base, mine, scale);
}

constexpr int kManyCols = 4;     // columns of a lane

// A wave's 64 rows of B (its columns' ranks) in LDS: 16-byte piece o of column
// CT i + c at 16 c + i rows of rank/8 pieces, o swizzled by i where a row is a
// power of two of them, so that 8 lanes' reads meet no bank twice.
template <int KS, int CT>
struct BTile {
  uint4 piece[16 * CT * 4 * KS];
};

// kAll: every piece requested at once (the start of a wave), or one after the
// other, which takes no registers from a tile under way (a later adapter).
template <bool kAll, int KS, int CT>
__device__ __forceinline__ void stage_b(const LoraArgs& p, int32_t a, int64_t wave_col, int lane,
                                        BTile<KS, CT>& t, int32_t mask, int32_t shift) {
  const int32_t per = p.rank / 8, count = 16 * CT * per;
  const int64_t left = (p.n - wave_col) * per - 1;   // the last piece that exists
  const uint4* b = reinterpret_cast<const uint4*>(
      p.b + (static_cast<int64_t>(a) * p.n + wave_col) * p.rank);
  wave_sync();
  const auto put = [&](int32_t e, uint4 v) {
    const int32_t col = e / per, o = e - col * per, i = col / CT, c = col % CT;
    t.piece[(16 * c + i) * per + (o ^ ((i >> shift) & mask))] = v;
  };
  if (kAll) {
    uint4 v[CT * KS];
#pragma unroll
    for (int j = 0; j < CT * KS; ++j)
      if (64 * j < count) v[j] = b[64 * j + lane < left ? 64 * j + lane : left];
#pragma unroll
    for (int j = 0; j < CT * KS; ++j)
      if (64 * j < count) put(64 * j + lane, v[j]);
  } else {
#pragma unroll 1
    for (int32_t e = lane; e < count; e += 64) put(e, b[e < left ? e : left]);
  }
  wave_sync();
}

// Waves a SIMD: as many as leave the registers of two tiles without spills.
template <int KS, int BK, int YK>
__global__ __launch_bounds__(256, KS > 2 ? 2 : BK == kNone || (KS == 1 && BK == kBf16) ? 4 : 3)
void expand_many_kernel(ExpandArgs s) {
  const LoraArgs& p = s.p;
  constexpr int CT = kManyCols;
  __shared__ BTile<KS, CT> tiles_b[4];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), i = lane & 15, g = lane >> 4;
  const uint32_t col_blocks = static_cast<uint32_t>((p.n + 64 * CT - 1) / (64 * CT));
  // row tiles major, columns minor, dealt to the XCDs as they come: a run of
  // neighbours on one XCD reads its adapters from one L2 but streams base and
  // y slower (108 against 101 us with the first product at 4096 rows, rank
  // 64, 16 adapters, 3840 -> 15360)
  const uint32_t unit = blockIdx.x;
  const uint32_t block_row = unit / col_blocks;
  const int64_t tile0 = static_cast<int64_t>(block_row) * s.tiles;
  const int64_t wave_col =
      (static_cast<int64_t>(unit - block_row * col_blocks) * 4 + wave) * (16 * CT);
  if (tile0 * 16 >= p.m || wave_col >= p.n) return;
  const bool full = wave_col + CT * i + CT <= p.n;
  const int32_t live =
      static_cast<int32_t>(p.m - tile0 * 16 < 16 * s.tiles ? p.m - tile0 * 16 : 16 * s.tiles);
  const int32_t per = p.rank / 8;
  const int32_t mask = (per & (per - 1)) == 0 ? (per < 8 ? per : 8) - 1 : 0;
  const int32_t shift = per >= 8 ? 0 : per == 4 ? 2 : 0;
  BTile<KS, CT>& bt = tiles_b[wave];
  int32_t loaded = -1;
  float sc = 1.0f;
  const int32_t count = (live + 15) / 16;
  const int64_t col = full ? wave_col + CT * i : p.n - CT;
  const auto rows_of = [&](int m) { return live - 16 * m < 16 ? live - 16 * m : 16; };
  // as loaded: looked at a tile later
  const auto load_id = [&](int m, int32_t& id) __attribute__((always_inline)) {
    if (p.ids != nullptr) id = p.ids[(tile0 + m) * 16 + (i < rows_of(m) ? i : 0)];
  };
  const auto adapter = [&](int32_t id, int32_t rows) __attribute__((always_inline)) {
    return i < rows && id >= 0 && id < p.n_adapters ? id : -1;
  };
  BaseTile<CT, BK> base0, base1;
  int32_t id0 = 0, id1 = 0;
  load_id(0, id0);
  load_base_any<CT, BK>(s, tile0 * 16, rows_of(0), g, col, base0);
  const int32_t first = adapter(id0, rows_of(0));
  const uint64_t any = __ballot(first >= 0);
  if (any != 0) {
    loaded = __builtin_amdgcn_readlane(first, __builtin_ctzll(any));
    sc = p.scale != nullptr ? p.scale[loaded] : 1.0f;
    stage_b<true, KS, CT>(p, loaded, wave_col, lane, bt, mask, shift);
  }
  // Tile m, whose base is on its way; the next one's (the last again behind the
  // end) is requested behind this one's operands, since loads return in order.
  // Two tiles' registers in turn: a copy would wait for the load.
  const auto step = [&](int m, const int32_t& raw, const BaseTile<CT, BK>& base_now,
                        int32_t& id_next, BaseTile<CT, BK>& base_next)
                        __attribute__((always_inline)) {
    const int64_t row0 = (tile0 + m) * 16;
    const int32_t rows = rows_of(m), next = m + 1 < count ? m + 1 : m;
    const int32_t id_now = adapter(raw, rows);
    load_id(next, id_next);
    uint4 hf[3][KS];
#pragma unroll
    for (int t = 0; t < 3; ++t)
#pragma unroll
      for (int k = 0; k < KS; ++k) hf[t][k] = s.frag[(((tile0 + m) * 3 + t) * KS + k) * 64 + lane];
    __builtin_amdgcn_sched_barrier(0);
    load_base_any<CT, BK>(s, (tile0 + next) * 16, rows_of(next), g, col, base_next);
    float scale[4];
    floatx4 mine[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) mine[c] = floatx4{0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q) scale[q] = -0.0f;
    uint32_t todo = static_cast<uint32_t>(__ballot(id_now >= 0)) & 0xFFFFu;
#pragma unroll 1
    while (todo != 0) {
      const int32_t a = __builtin_amdgcn_readlane(id_now, __builtin_ctz(todo));
      const uint32_t match = static_cast<uint32_t>(__ballot(id_now == a)) & 0xFFFFu;
      todo &= ~match;
      if (a != loaded) {
        loaded = a;
        sc = p.scale != nullptr ? p.scale[a] : 1.0f;
        stage_b<false, KS, CT>(p, a, wave_col, lane, bt, mask, shift);
        asm volatile("" : "+v"(sc));   // waited for here, not by every tile
      }
      floatx4 acc[CT];
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[c] = floatx4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint4 bf[CT];
        const int32_t o = 4 * k + g;
        const bool ok = o < per;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          bf[c] = bt.piece[(16 * c + i) * per + ((ok ? o : 0) ^ ((i >> shift) & mask))];
          if (32 * k + 32 > p.rank) {
            bf[c].x = ok ? bf[c].x : 0u;
            bf[c].y = ok ? bf[c].y : 0u;
            bf[c].z = ok ? bf[c].z : 0u;
            bf[c].w = ok ? bf[c].w : 0u;
          }
        }
#pragma unroll
        for (int t = 0; t < 3; ++t)
#pragma unroll
          for (int c = 0; c < CT; ++c)
            acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(hf[t][k]), as_bf16x8(bf[c]),
                                                             acc[c], 0, 0, 0);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool hit = (match >> (4 * g + q)) & 1u;
        scale[q] = hit ? sc : scale[q];
#pragma unroll
        for (int c = 0; c < CT; ++c) mine[c][q] = hit ? acc[c][q] : mine[c][q];
      }
    }
    redo_nan(p, id_now, wave_col, lane, mine, [&](int t, int32_t r) {
      const uint16_t* term = reinterpret_cast<const uint16_t*>(
          s.frag + ((tile0 + m) * 3 * KS + r / 32) * 64 + 16 * (r % 32 / 8) + t) + r % 8;
      return (bf16_f32(term[0]) + bf16_f32(term[KS * 512])) + bf16_f32(term[2 * KS * 512]);
    });
    finish_rows<CT, BK, YK>(s, row0, rows, g, wave_col, CT * i, full, base_now, mine, scale);
  };
  int32_t m = 0;
#pragma unroll 1
  for (; m + 1 < count; m += 2) {
    step(m, id0, base0, id1, base1);
    step(m + 1, id1, base1, id0, base0);
  }
  if (m < count) step(m, id0, base0, id1, base1);
}

int32_t slices_of(int64_t k) { return static_cast<int32_t>((k + kSlice - 1) / kSlice); }

// Whether the many-rows product does: one adapter, 4096 columns of rank 16, 512
// rows 10.1 us and 13.4 by few rows (256: 9.4 and 9.0), 128 rows of 15360 10.1
// and 13.0. Several adapters may be mixed in every tile, which only the few-rows
// kernels deal to waves: 256 rows of 15360 columns, rank 64, 16 adapters in runs
// 37 and 34, 512 rows 41 and 51, so these ask for more rows.
bool many_rows(int64_t m, int64_t n, bool one_adapter) {
  if (n < kManyCols) return false;
  return one_adapter ? m >= 128 && m * n >= (1 << 21) : m >= 512 && m * n >= (1 << 22);
}

// Grain of the first product before the few-rows one: partial sums it leaves
// per value. 61 rows of 32 adapters, rank 32, 15360 -> 3840: both products 21 us
// in slices, 44 in running sums; 700 rows of one, rank 64, 15360 -> 1024: 37 and
// 24.
int32_t shrink_parts(int64_t m, int64_t k) {
  const int64_t tiles = (m + 15) / 16;
  const int32_t slices = slices_of(k);
  return tiles * kStreams >= 256 && slices > kStreams ? kStreams : slices;
}

// Bytes of h as operands of the many-rows product.
int64_t frag_bytes(int64_t m, int32_t rank) {
  return (m + 15) / 16 * 3 * ((rank + 31) / 32) * 1024;
}

// Whether one launch does (see one_pass_kernel): at most two adapters whose A
// is small. In a captured graph one row of rank 16, 3840 -> 15360, takes 6.4 us
// (two launches: 8.1), 15360 -> 3840 9.3 (9.9), 16 rows of two adapters of rank
// 32, 512 -> 8192, 7.1 (9.5); eight rows of eight adapters of rank 16, 4096 ->
// 4096, would take 18.8 (10.7).
bool one_pass(int64_t m, int64_t k, int32_t rank, int32_t n_adapters, bool mixed) {
  const int64_t adapters = !mixed ? 1 : m < n_adapters ? m : n_adapters;
  return m <= 16 && rank <= 32 && adapters <= 2 && rank * k * adapters <= 262144;
}

template <int RT, int BK, int YK>
void launch_one_shape(const ShrinkArgs& sh, const ExpandArgs& s, hipStream_t st) {
  hipLaunchKernelGGL((one_pass_kernel<RT, BK, YK>),
                     dim3(static_cast<uint32_t>((s.p.n + 255) / 256)), dim3(512), 0, st, sh, s);
}

template <int RT>
void launch_one_ranks(const ShrinkArgs& sh, const ExpandArgs& s, hipStream_t st) {
  switch (s.base_kind * 2 + (s.y_bf16 ? 1 : 0)) {
    case 0: return launch_one_shape<RT, kNone, kF32>(sh, s, st);
    case 1: return launch_one_shape<RT, kNone, kBf16>(sh, s, st);
    case 2: return launch_one_shape<RT, kF32, kF32>(sh, s, st);
    case 3: return launch_one_shape<RT, kF32, kBf16>(sh, s, st);
    case 4: return launch_one_shape<RT, kBf16, kF32>(sh, s, st);
    default: return launch_one_shape<RT, kBf16, kBf16>(sh, s, st);
  }
}

int64_t add_workspace(int64_t m, int64_t n, int64_t k, int32_t rank) {
  if (m == 1 && one_pass(m, k, rank, 1, false)) return 0;
  const int64_t few = shrink_parts(m, k) * m * rank * 4, many = frag_bytes(m, rank);
  if (many_rows(m, n, false)) return many;
  return many_rows(m, n, true) && many > few ? many : few;
}

template <bool kAny>
void launch_shrink(const ShrinkArgs& s, hipStream_t st) {
  const LoraArgs& p = s.p;
  const dim3 grid = xcd_grid(s.tiles * s.parts);
  const int64_t mixed = p.ids == nullptr || s.perm != nullptr ? 1
                        : p.m < p.n_adapters                  ? p.m
                                                              : p.n_adapters;
  uint32_t threads = s.frag != nullptr ? 64 * kStreams : mixed < 2 ? 64 : mixed < 8 ? 256 : 512;
  // a grid ends below 2^32 threads (2^24 rows in 8 running sums have 2^23
  // blocks); any number of waves can be dealt a tile's adapters
  if (static_cast<uint64_t>(grid.x) * threads > 0xFFFFFFFFull) threads = 256;
  const dim3 block(threads);
  if (p.rank <= 16) hipLaunchKernelGGL((shrink_kernel<1, kAny>), grid, block, 0, st, s);
  else if (p.rank <= 32) hipLaunchKernelGGL((shrink_kernel<2, kAny>), grid, block, 0, st, s);
  else if (p.rank <= 64) hipLaunchKernelGGL((shrink_kernel<4, kAny>), grid, block, 0, st, s);
  else hipLaunchKernelGGL((shrink_kernel<8, kAny>), grid, block, 0, st, s);
}

template <int KS, int BK, int YK>
void launch_expand_shape(ExpandArgs s, hipStream_t st) {
  const int64_t m = s.p.m, n = s.p.n;
  if (s.frag != nullptr) {
    // up to eight tiles a block while the blocks fill the chip: 2048 rows, 4096
    // columns, rank 16: 26 us with eight, 19 with two
    const int64_t tiles = (m + 15) / 16, cols = (n + 64 * kManyCols - 1) / (64 * kManyCols);
    s.tiles = 8;
    while (s.tiles > 1 && (tiles + s.tiles - 1) / s.tiles * cols < 768) s.tiles /= 2;
    hipLaunchKernelGGL((expand_many_kernel<KS, BK, YK>),
                       dim3(static_cast<uint32_t>(cols * ((tiles + s.tiles - 1) / s.tiles))),
                       dim3(256), 0, st, s);
  } else {
    hipLaunchKernelGGL((expand_few_kernel<KS, BK, YK>),
                       xcd_grid((n + 127) / 128 * ((m + 15) / 16)), dim3(256), 0, st, s);
  }
}

template <int KS>
void launch_expand_ranks(const ExpandArgs& s, hipStream_t st) {
  switch (s.base_kind * 2 + (s.y_bf16 ? 1 : 0)) {
    case 0: return launch_expand_shape<KS, kNone, kF32>(s, st);
    case 1: return launch_expand_shape<KS, kNone, kBf16>(s, st);
    case 2: return launch_expand_shape<KS, kF32, kF32>(s, st);
    case 3: return launch_expand_shape<KS, kF32, kBf16>(s, st);
    case 4: return launch_expand_shape<KS, kBf16, kF32>(s, st);
    default: return launch_expand_shape<KS, kBf16, kBf16>(s, st);
  }
}

void launch_expand(const ExpandArgs& s, hipStream_t st) {
  if (s.p.rank <= 32) launch_expand_ranks<1>(s, st);
  else if (s.p.rank <= 64) launch_expand_ranks<2>(s, st);
  else if (s.p.rank <= 96) launch_expand_ranks<3>(s, st);
  else launch_expand_ranks<4>(s, st);
}

// --------------------------------------------------------------- backward
// With Bt and At, B and A turned round (a small copy), the two products of
// the forward give g = Bt dy and dx = dx_base + s At g. What is new is the
// sum over rows, dA = s g^T x and dB = s h^T dy:
//  - prepare_kernel makes Bt and At and sorts the rows by adapter, each
//    adapter's from a multiple of 32 rows on (ids NULL: rows as they are);
//  - outer_kernel: a wave has 128 columns of x or dy, 16 ranks and a range of
//    tiles. A lane loads 8 columns of 8 rows and turns the 8 x 8
//    block with v_perm, which makes the operand whose K is the rows; the other
//    operand is g or h of these rows in three bf16 terms; sums stay in
//    registers until the adapter changes. An adapter inside one range is
//    written at once, one over several leaves a partial sum in each;
//  - reduce_kernel adds those in range order and writes zeros for adapters
//    without rows. Few rows (a matter of launches) do without it: there a wave
//    has all tiles of one adapter.
// Rows of another adapter never meet in one MFMA chain.
// g runs over the sorted rows too, so that none of its tiles is mixed (2048
// rows of 8 adapters at random, rank 32, 4096 -> 4096: the call 86 -> 62 us).
// A large dy of one rank chunk is read once, g's sums beside dB's (join_kernel
// adds them), in a launch of its own; else g is the first product on Bt.
// Measured, 8192 rows, 15360 and 3840 columns, one adapter of rank 16: prepare
// 4.8 us, dy 68.3 (252 MB, 3.7 TB/s: a CU has some 75 lines under way, which
// its L1 allows, for 1300 clocks each), join 6.7, dx 28.2 (126 MB), x 16.6,
// reduce 6.8; with dy read twice 55.6 for g and 70.4 for both sums.
constexpr int kMaxSorted = 4096;       // adapters prepare_kernel counts in LDS

struct TurnArgs {
  const uint16_t* from;
  uint16_t* to;
  int64_t rows, cols, rows_pad;     // from [rows][cols] -> to [cols][rows_pad] per adapter
  int32_t n_adapters;
};

// 8 rows of 8 bf16 -> 8 columns of 8.
__device__ __forceinline__ void turn_block(const uint4 (&v)[8], uint4 (&t)[8]) {
  uint32_t d[8][4];
  __builtin_memcpy(d, v, 128);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo[j] = vperm(d[2 * j + 1][c], d[2 * j][c], 0x05040100u);
      hi[j] = vperm(d[2 * j + 1][c], d[2 * j][c], 0x07060302u);
    }
    t[2 * c] = uint4{lo[0], lo[1], lo[2], lo[3]};
    t[2 * c + 1] = uint4{hi[0], hi[1], hi[2], hi[3]};
  }
}

// Blocks of 8 x 8, one a thread: B's in order of rows (stores coalesced), A's
// in order of columns.
__device__ __forceinline__ int64_t turn_count(const TurnArgs& p) {
  return p.n_adapters * (p.rows_pad / 8) * (p.cols / 8);
}

__device__ __forceinline__ void turn_matrices(const TurnArgs& b, const TurnArgs& a, int64_t e) {
  const int64_t nb = turn_count(b);
  const bool first = e < nb;
  const TurnArgs& p = first ? b : a;
  if (!first) e -= nb;
  const int64_t rb = p.rows_pad / 8, cb = p.cols / 8;
  const int64_t i = e / (rb * cb), at = e - i * rb * cb;
  const int64_t r = 8 * (first ? at % rb : at / cb), c = 8 * (first ? at / rb : at % cb);
  uint4 v[8], t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = r + j < p.rows
               ? *reinterpret_cast<const uint4*>(p.from + (i * p.rows + r + j) * p.cols + c)
               : uint4{0, 0, 0, 0};
  turn_block(v, t);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4*>(p.to + (i * p.cols + c + j) * p.rows_pad + r) = t[j];
}

// Where sorted rows lie.
struct Order {
  const int32_t* perm;     // [tiles * 32] row or -1; NULL: rows as they are, all adapter 0
  const int32_t* adapter;  // [tiles]
  const int32_t* tile0;    // [n_adapters + 1] first tile of each adapter
  int32_t tiles;           // perm NULL: their number
};

__device__ __forceinline__ int32_t first_tile(const Order& o, int32_t a) {
  return o.perm != nullptr ? o.tile0[a] : a == 0 ? 0 : o.tiles;
}

constexpr int kSortStep = 8;   // rows a thread looks at together

// The ids of rows t to t + 7 as they are; -1 behind the last.
__device__ __forceinline__ void load_ids(const LoraArgs& p, int64_t t, int32_t (&ids)[kSortStep]) {
  if (t + kSortStep <= p.m) {
    __builtin_memcpy(ids, p.ids + t, sizeof(ids));
    return;
  }
#pragma unroll
  for (int j = 0; j < kSortStep; ++j) ids[j] = t + j < p.m ? p.ids[t + j] : -1;
}

// A block of 512 collects the rows of adapter a in rising order, behind the
// tiles of the adapters before it.
__device__ void order_rows(const LoraArgs& p, int32_t a, int32_t* perm, int32_t* adapter,
                           int32_t* tile0) {
  __shared__ int32_t counts[kMaxSorted];
  __shared__ int32_t sums[8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int32_t e = threadIdx.x; e <= a && e < p.n_adapters; e += 512) counts[e] = 0;
  __syncthreads();
  int32_t ids[kSortStep], next[kSortStep];
  const int64_t mine0 = kSortStep * threadIdx.x;
  load_ids(p, mine0, next);
  for (int64_t t0 = 0; t0 < p.m; t0 += 512 * kSortStep) {
#pragma unroll
    for (int j = 0; j < kSortStep; ++j) ids[j] = next[j];
    load_ids(p, t0 + 512 * kSortStep + mine0, next);
#pragma unroll
    for (int j = 0; j < kSortStep; ++j) {
      const int32_t id = ids[j], one = __builtin_amdgcn_readfirstlane(id);
      if (__ballot(id == one) == ~0ull) {   // a run of one adapter: one count
        if (lane == 0 && one >= 0 && one <= a) atomicAdd(&counts[one], 64);
      } else if (id >= 0 && id <= a) {
        atomicAdd(&counts[id], 1);
      }
    }
  }
  __syncthreads();
  int32_t before = 0;
  for (int32_t e = threadIdx.x; e < a; e += 512) before += (counts[e] + kRowTile - 1) / kRowTile;
  for (int q = 32; q >= 1; q >>= 1) before += __shfl_xor(before, q, 64);
  if (lane == 0) sums[wave] = before;
  __syncthreads();
  before = 0;
  for (int w = 0; w < 8; ++w) before += sums[w];
  const int32_t mine = counts[a], tiles = (mine + kRowTile - 1) / kRowTile;
  if (threadIdx.x == 0) {
    tile0[a] = before;
    if (a == p.n_adapters - 1) tile0[a + 1] = before + tiles;
  }
  for (int32_t e = threadIdx.x; e < tiles; e += 512) adapter[before + e] = a;
  perm += static_cast<int64_t>(before) * kRowTile;
  for (int32_t e = mine + threadIdx.x; e < tiles * kRowTile; e += 512) perm[e] = -1;
  // kSortStep neighbouring rows a thread
  int32_t at = 0;
  load_ids(p, mine0, next);
  for (int64_t t0 = 0; t0 < p.m && at < mine; t0 += 512 * kSortStep) {
    const int64_t t = t0 + mine0;
    int32_t ahead = 0, all = 0;
#pragma unroll
    for (int j = 0; j < kSortStep; ++j) ids[j] = next[j];
    load_ids(p, t + 512 * kSortStep, next);
#pragma unroll
    for (int j = 0; j < kSortStep; ++j) {
      const uint64_t hits = __ballot(ids[j] == a);
      ahead += __builtin_popcountll(hits & ((1ull << lane) - 1));
      all += __builtin_popcountll(hits);
    }
    __syncthreads();
    if (lane == 0) sums[wave] = all;
    __syncthreads();
    int32_t off = at + ahead;
    for (int w = 0; w < 8; ++w) {
      if (w < wave) off += sums[w];
      at += sums[w];
    }
#pragma unroll
    for (int j = 0; j < kSortStep; ++j)
      if (ids[j] == a) perm[off++] = static_cast<int32_t>(t + j);
  }
}

struct OuterSide {
  const uint16_t* s;       // rows [m][wide]
  const float* v;          // g or h, [m][rank]
  void* grad;
  float* part;             // [2 * splits][rank * cols]
  int64_t ld, cols, wide;  // wide: cols, or 8 where fewer (zeros behind them)
  int32_t blocks;          // of four waves, a split (0: not in this launch)
  int32_t per_split;       // tiles of a split; 0: a split is an adapter
};

struct OuterArgs {
  OuterSide side[2];       // 0: x and g -> dA [rank][cols]; 1: dy and h -> dB [cols][rank]
  Order o;
  const float* scale;
  int64_t m;
  int32_t rank, n_adapters;
  bool grad_bf16;
  const uint16_t* bt;      // kSums: [n_adapters][rank][n_pad]
  float* sums;             // [blocks][tiles][32][16]
  int64_t n_pad, tiles;
};

// v moved down by n of its 8 elements (1..8), zeros behind.
__device__ __forceinline__ uint4 shift8(uint4 v, int n) {
  const uint32_t d[4] = {v.x, v.y, v.z, v.w};
  uint32_t w[5];
#pragma unroll
  for (int j = 0; j < 5; ++j) {
    w[j] = 0;
#pragma unroll
    for (int q = 0; q + j < 4; ++q) w[j] = (n >> 1) == q ? d[q + j] : w[j];
  }
  if (n & 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = (w[j] >> 16) | (w[j + 1] << 16);
  }
  return uint4{w[0], w[1], w[2], w[3]};
}

// A wave: 128 columns, 16 ranks, a split's tiles. A block's waves take the
// rank chunks of the same columns side by side, so that these meet in the L1.
//
// kSums (one rank chunk, dy alone): the block also leaves what its 512 columns
// add to g = Bt dy, so that dy is read once. The rows as loaded go through LDS
// into operands whose K is the columns.
template <bool kSums, bool kSorted>
__global__ __launch_bounds__(256, 2) void outer_kernel(OuterArgs p) {
  __shared__ uint4 loaded[kSums ? 4 : 1][kSums ? 512 : 1];
  __shared__ float sums[4][kSums ? 4 : 1][kSums ? 640 : 1];   // row r, rank i at 16 (r + r / 4) + i
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), i = lane & 15, g = lane >> 4;
  const int32_t per = p.side[0].blocks + p.side[1].blocks;
  // a range of tiles, or an adapter
  const int32_t split = blockIdx.x / per, at = blockIdx.x - split * per;
  const bool second = at >= p.side[0].blocks;
  // picked one by one: through an indexed struct the compiler would lose that
  // the pointers are global ones, and wait for every load (flat) at once
  const char* const rows_in = reinterpret_cast<const char*>(second ? p.side[1].s : p.side[0].s);
  const char* const vectors = reinterpret_cast<const char*>(second ? p.side[1].v : p.side[0].v);
  const uint32_t row_bytes = static_cast<uint32_t>(second ? p.side[1].ld : p.side[0].ld) * 2;
  const uint32_t vector_bytes = p.rank * 4;
  const int64_t cols = second ? p.side[1].cols : p.side[0].cols;
  const int64_t wide = second ? p.side[1].wide : p.side[0].wide;
  const int64_t group = second ? at - p.side[0].blocks : at;   // kSums
  const int32_t chunks = (p.rank + 15) / 16;
  const int32_t job = (second ? at - p.side[0].blocks : at) * 4 + wave, chunk = job % chunks;
  const int64_t col0 = static_cast<int64_t>(job / chunks) * 128;
  if (!kSums && col0 >= cols) return;   // with kSums the wave adds zeros: the block meets
  const bool whole = col0 + 128 <= wide;
  // a row's last piece is loaded as its last 8 columns and moved down
  const int64_t col = col0 + 8 * i, over = col + 8 - wide;
  const int shift = over <= 0 ? 0 : over < 8 ? static_cast<int>(over) : 8;
  const uint32_t offset0 = static_cast<uint32_t>(over <= 0 ? col : wide - 8) * 2;
  const uint32_t offset = offset0 + 8 * g * row_bytes;
  const char* const from = rows_in + offset0;
  const int32_t per_split = second ? p.side[1].per_split : p.side[0].per_split;
  const bool by_adapter = per_split == 0;
  const int32_t n_tiles = first_tile(p.o, p.n_adapters);
  const int32_t begin = by_adapter ? first_tile(p.o, split) : split * per_split;
  const int32_t end = by_adapter                        ? first_tile(p.o, split + 1)
                      : begin + per_split < n_tiles ? begin + per_split
                                                      : n_tiles;
  if (begin >= end && !by_adapter) return;

  floatx4 acc[8];
  // The sums' NaN of one adapter's tiles t0 to t1 again from the values, as in
  // redo_nan: an infinite row value beside a v of fewer than three terms.
  const auto redo = [&](int32_t t0, int32_t t1) __attribute__((always_inline)) {
    int32_t own = lane;
    asm volatile("" : "+v"(own));
    const int32_t rank = 16 * chunk + (own & 15);
    constexpr int kAhead = 4;   // rows on their way at once, of a tile
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t cc = col0 + 8 * (4 * (own >> 4) + q);
      bool open = false;
#pragma unroll
      for (int c = 0; c < 8; ++c) open |= cc + c < cols && is_nan(acc[c][q]);
      if (rank >= p.rank || !open) continue;
      float sum[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[c] = 0.0f;
#pragma unroll 1
      for (int64_t e = static_cast<int64_t>(t0) * kRowTile;
           e < static_cast<int64_t>(t1) * kRowTile && open; e += kAhead) {
        float v[kAhead];
        uint32_t d[kAhead][4];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int64_t row = kSorted ? p.o.perm[e + j] : e + j < p.m ? e + j : -1;
          const int64_t at = row < 0 ? 0 : row;   // behind the adapter's last: zeros
          const uint4 piece = load8_part(
              reinterpret_cast<const uint16_t*>(rows_in + at * row_bytes) + cc, cols - cc);
          v[j] = *reinterpret_cast<const float*>(vectors + at * vector_bytes + 4 * rank);
          __builtin_memcpy(d[j], &piece, 16);
          if (row < 0) v[j] = 0.0f, d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0;
        }
        open = false;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            sum[c] = __builtin_fmaf(v[j], c & 1 ? bf16_hi(d[j][c / 2]) : bf16_lo(d[j][c / 2]),
                                    sum[c]);
          open |= !is_nan(sum[c]);
        }
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c][q] = is_nan(acc[c][q]) ? sum[c] : acc[c][q];
    }
  };
  const auto flush = [&](int32_t a, int32_t t0, int32_t t1) __attribute__((always_inline)) {
    if (__ballot(any_nan(acc)) != 0) redo(t0, t1);
    // kept from being computed ahead of the loop and held through it
    int32_t own = lane;
    asm volatile("" : "+v"(own));
    const int i = own & 15, g = own >> 4;
    const int32_t s0 = first_tile(p.o, a), s1 = first_tile(p.o, a + 1);
    const bool direct = by_adapter || (s0 >= begin && s1 <= begin + per_split);
    const int64_t size = p.rank * cols;
    // an adapter without rows gets zeros, whatever its scale
    const float f = !direct || p.scale == nullptr || s0 == s1 ? 1.0f : p.scale[a];
    void* const grad = second ? p.side[1].grad : p.side[0].grad;
    float* const part = second ? p.side[1].part : p.side[0].part;
    void* to = direct ? grad : static_cast<void*>(part);
    const int64_t base = direct ? a * size : (2 * split + (s0 < begin ? 0 : 1)) * size;
    const bool bf16 = direct && p.grad_bf16;
    const int32_t rank = 16 * chunk + i;
    if (rank >= p.rank) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t cc = col0 + 8 * (4 * g + q);
      if (!second) {
        if (cc >= cols) continue;
        const int64_t e = base + rank * cols + cc;
        if (bf16) {
          uint32_t d[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) d[c] = pack_bf16(f * acc[2 * c][q], f * acc[2 * c + 1][q]);
          __builtin_memcpy(static_cast<uint16_t*>(to) + e, d, 16);
        } else {
          float d[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) d[c] = f * acc[c][q];
          __builtin_memcpy(static_cast<float*>(to) + e, d, 32);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (cc + c < cols) store_any(to, base + (cc + c) * p.rank + rank, bf16, f * acc[c][q]);
      }
    }
  };

  // One adapter's tiles at a time. Two tiles are on their way while one is
  // multiplied, and the rows of the one to be requested next are known (their
  // numbers are a load of their own, sent before the tile's: loads return in
  // order). Every request is made, the last tile's again behind the end: a
  // conditional one would leave the compiler to wait for all loads instead of
  // the oldest ones.
  uint4 bt[4];
  int32_t buffer = 0;   // of sums: two tiles' at a time
  const int32_t my_rank = 16 * chunk + i < p.rank ? 16 * chunk + i : p.rank - 1;
  int32_t tile = begin;
  do {
    const int32_t a = by_adapter ? split : kSorted ? uniform(p.o.adapter[tile]) : 0;
    const int32_t a_end = by_adapter ? end : first_tile(p.o, a + 1), stop = a_end < end ? a_end : end;
    const int32_t start = tile;
    uint4 in0[8], in1[8];
    float v0[8], v1[8];
    int32_t rows[8], miss0, miss1;
    const auto find = [&](int32_t t) __attribute__((always_inline)) {
      if (!kSorted) return;
      t = t < stop ? t : stop - 1;
      const int4* at =
          reinterpret_cast<const int4*>(p.o.perm + static_cast<int64_t>(t) * kRowTile + 8 * g);
      const int4 lo = at[0], hi = at[1];
      rows[0] = lo.x, rows[1] = lo.y, rows[2] = lo.z, rows[3] = lo.w;
      rows[4] = hi.x, rows[5] = hi.y, rows[6] = hi.z, rows[7] = hi.w;
    };
    // tile t, whose rows were found last, then the search for the next one's.
    // Rows as they are lie at 32-bit offsets from the tile's first (strides are
    // at most 2^24), others at a 64-bit product each.
    const auto request = [&](int32_t t, uint4 (&to)[8], float (&v)[8],
                             int32_t& mask) __attribute__((always_inline)) {
      mask = 0;
      if (kSorted) {
        int32_t now[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) now[j] = rows[j];
        find(t + 1);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint64_t row = now[j] < 0 ? 0 : now[j];
          mask |= now[j] < 0 ? 1 << j : 0;
          to[j] = load8(reinterpret_cast<const uint16_t*>(from + row * row_bytes));
          v[j] = *reinterpret_cast<const float*>(vectors + row * vector_bytes + 4 * my_rank);
        }
      } else {
        t = t < stop ? t : stop - 1;
        const char* const tile_rows = rows_in + static_cast<int64_t>(t) * kRowTile * row_bytes;
        const char* const tile_vectors = vectors + static_cast<int64_t>(t) * kRowTile * vector_bytes;
        const int64_t left = p.m - static_cast<int64_t>(t) * kRowTile;
        uint32_t r[8], d[8], r0 = offset, d0 = 8 * g * vector_bytes + 4 * my_rank;
        asm volatile("" : "+v"(r0), "+v"(d0));   // the others are no registers through the loop
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          r[j] = r0 + j * row_bytes;
          d[j] = d0 + j * vector_bytes;
        }
        if (left < kRowTile) {   // its last row again in place of those behind it
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t row = 8 * g + j < left ? 8 * g + j : static_cast<uint32_t>(left) - 1;
            mask |= 8 * g + j < left ? 0 : 1 << j;
            r[j] = offset0 + row * row_bytes;
            d[j] = row * vector_bytes + 4 * my_rank;
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          to[j] = load8(reinterpret_cast<const uint16_t*>(tile_rows + r[j]));
          v[j] = *reinterpret_cast<const float*>(tile_vectors + d[j]);
        }
      }
    };
    const auto multiply = [&](int32_t t, uint4 (&in)[8], float (&vi)[8],
                              int32_t& mask) __attribute__((always_inline)) {
      uint4 rows_in[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) rows_in[j] = in[j], w[j] = vi[j];
      if (!whole && shift != 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) rows_in[j] = shift8(in[j], shift);
      }
      if (__ballot(mask != 0) != 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (mask >> j & 1) rows_in[j] = uint4{0, 0, 0, 0}, w[j] = 0.0f;
      }
      uint4 st[8], v[3];
      if (kSums) {
#pragma unroll
        for (int j = 0; j < 8; ++j) loaded[wave][16 * (8 * g + j) + (i ^ j)] = rows_in[j];
      }
      turn_block(rows_in, st);
      uint16_t d[3][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) split3(w[j], d[0][j], d[1][j], d[2][j]);
#pragma unroll
      for (int k = 0; k < 3; ++k) v[k] = __builtin_bit_cast(uint4, d[k]);
      // what was loaded is used up by now: a last use behind the request would
      // have it take other registers, and their copy back wait for the loads
#pragma unroll
      for (int k = 0; k < 3; ++k)
        asm volatile("" : "+v"(v[k].x), "+v"(v[k].y), "+v"(v[k].z), "+v"(v[k].w));
      request(t + 2, in, vi, mask);
      if (kSums) {
        wave_sync();
        floatx4 add[2] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            add[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                as_bf16x8(loaded[wave][16 * (16 * h + i) + ((4 * k + g) ^ (i & 7))]),
                as_bf16x8(bt[k]), add[h], 0, 0, 0);
        float* mine = sums[buffer][wave];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < 4; ++q) mine[16 * (20 * h + 5 * g + q) + i] = add[h][q];
        buffer = (buffer + 1) & 3;
      }
#pragma unroll
      for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int c = 0; c < 8; ++c)
          acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(st[c]), as_bf16x8(v[q]),
                                                           acc[c], 0, 0, 0);
    };
    // the block's sum of tile t
    const auto join = [&](int32_t t, int32_t from) __attribute__((always_inline)) {
      const int row = threadIdx.x >> 3, at = 16 * (row + (row >> 2)) + 2 * (threadIdx.x & 7);
      float2 d = *reinterpret_cast<const float2*>(&sums[from][0][at]);
#pragma unroll
      for (int w = 1; w < 4; ++w) {
        const float2 e = *reinterpret_cast<const float2*>(&sums[from][kSums ? w : 0][at]);
        d.x += e.x, d.y += e.y;
      }
      reinterpret_cast<float2*>(p.sums)[(group * p.tiles + t) * 256 + threadIdx.x] = d;
    };
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = floatx4{0, 0, 0, 0};
    if (kSums) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t c = col0 + 32 * k + 8 * g;
        bt[k] = i < p.rank && c < p.n_pad
                    ? *reinterpret_cast<const uint4*>(p.bt + (static_cast<int64_t>(a) * p.rank + i) *
                                                                 p.n_pad + c)
                    : uint4{0, 0, 0, 0};
      }
    }
    if (tile < stop) {
      find(tile);
      request(tile, in0, v0, miss0);
      __builtin_amdgcn_sched_barrier(0);   // in this order also here
      request(tile + 1, in1, v1, miss1);
      __builtin_amdgcn_sched_barrier(0);
      // (an odd last tile is not a second one under a condition: the compiler
      // would wait for both tiles' loads)
#pragma unroll 1
      for (; tile + 1 < stop; tile += 2) {
        multiply(tile, in0, v0, miss0);
        multiply(tile + 1, in1, v1, miss1);
        if (kSums) {
          // two buffers of two: who writes one again has met all who read it
          lds_barrier();
          join(tile, buffer ^ 2);
          join(tile + 1, (buffer ^ 2) + 1);
        }
      }
      if (tile < stop) {
        multiply(tile, in0, v0, miss0);
        if (kSums) {
          buffer = (buffer + 1) & 3;
          lds_barrier();
          join(tile, buffer ^ 2);
        }
      }
      tile = stop;
    }
    flush(a, start, stop);   // an adapter without rows: zeros
  } while (tile < end);
}

// The blocks' sums of g (outer_kernel, kSums) in their order, four ranks of a
// sorted row a thread: as fp32 and as the operands of dx's product.
struct JoinArgs {
  LoraArgs p;
  Order o;
  const float* sums;
  float* g;
  uint4* frag;             // or NULL
  int64_t tiles;
  int32_t blocks;
};

__global__ __launch_bounds__(256) void join_kernel(JoinArgs s) {
  const LoraArgs& p = s.p;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, at = e >> 2;
  const int quad = static_cast<int>(e & 3);
  if (p.ids != nullptr && p.status != nullptr && e < p.m && p.ids[e] != -1 && adapter_of(p, e) < 0)
    atomicOr(p.status, static_cast<uint32_t>(BINADE_DEV_BAD_INDEX));
  if (at >= static_cast<int64_t>(first_tile(s.o, p.n_adapters)) * kRowTile) return;
  const int64_t row = s.o.perm != nullptr ? s.o.perm[at] : at < p.m ? at : -1;
  if (row < 0) return;
  const floatx4* from = reinterpret_cast<const floatx4*>(s.sums) + e;
  floatx4 v{0, 0, 0, 0};
#pragma unroll 8
  for (int32_t b = 0; b < s.blocks; ++b) v += from[b * s.tiles * (kRowTile * 4)];
  if (4 * quad < p.rank) *reinterpret_cast<floatx4*>(s.g + row * p.rank + 4 * quad) = v;
  if (s.frag == nullptr) return;
  // ranks behind the last meet zeros of At: an infinite dy has made them NaN
  if (4 * quad >= p.rank) v = floatx4{0, 0, 0, 0};
  uint16_t d[3][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) split3(v[j], d[0][j], d[1][j], d[2][j]);
  // ranks 8 (quad / 2) on of the row; zeros 16 ranks further
  uint4* to = s.frag + row / 16 * 192 + 16 * (quad >> 1) + row % 16;
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    reinterpret_cast<uint2*>(to + 64 * t)[quad & 1] = __builtin_bit_cast(uint2, d[t]);
    reinterpret_cast<uint2*>(to + 64 * t + 32)[quad & 1] = uint2{0, 0};
  }
}

// The first sort_blocks blocks: sorted rows of an adapter each; the others:
// Bt and At, by one wave a block (600 rows of 24 adapters of rank 64, 15360 x
// 3840: the call 158 us, with eight waves 181).
struct PrepareArgs {
  LoraArgs p;
  TurnArgs tb, ta;
  int32_t *perm, *adapter, *tile0;
  int32_t sort_blocks;
  int64_t turns;
};

__global__ __launch_bounds__(512) void prepare_kernel(PrepareArgs s) {
  const int32_t at = blockIdx.x;
  if (at < s.sort_blocks)
    order_rows(s.p, at, s.perm, s.adapter, s.tile0);
  else if (threadIdx.x < 64)
    for (int64_t e = static_cast<int64_t>(at - s.sort_blocks) * 64 + threadIdx.x; e < s.turns;
         e += static_cast<int64_t>(gridDim.x - s.sort_blocks) * 64)
      turn_matrices(s.tb, s.ta, e);
}

// dy with fewer than 8 columns, zeros behind them.
__global__ __launch_bounds__(256) void widen_kernel(const uint16_t* from, int64_t ld, int64_t cols,
                                                    int64_t m, uint16_t* to) {
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (e >= 8 * m) return;
  to[e] = e % 8 < cols ? from[e / 8 * ld + e % 8] : static_cast<uint16_t>(0);
}

// Four values of a gradient a thread; blockIdx.y: adapter.
__global__ __launch_bounds__(256) void reduce_kernel(OuterArgs p) {
  const int32_t a = blockIdx.y;
  const int64_t size[2] = {p.rank * p.side[0].cols, p.rank * p.side[1].cols};
  int64_t e = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (e >= size[0] + size[1]) return;
  const int side = e >= size[0] ? 1 : 0;
  if (side) e -= size[0];
  const int32_t s0 = first_tile(p.o, a), s1 = first_tile(p.o, a + 1);
  const int32_t per = p.side[side].per_split;
  const int32_t q0 = s0 / per, q1 = s1 > s0 ? (s1 - 1) / per : q0;
  if (s1 > s0 && q0 == q1) return;   // outer_kernel wrote it
  floatx4 v{0, 0, 0, 0};
  if (s1 > s0) {
    const float* part = p.side[side].part + e;
    v = *reinterpret_cast<const floatx4*>(part + (2 * q0 + 1) * size[side]);
#pragma unroll 8
    for (int32_t q = q0 + 1; q <= q1; ++q)
      v += *reinterpret_cast<const floatx4*>(part + 2 * q * size[side]);
    const float f = p.scale != nullptr ? p.scale[a] : 1.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= f;
  }
  const int64_t at = a * size[side] + e;
  if (p.grad_bf16) {
    const uint32_t d[2] = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    __builtin_memcpy(static_cast<uint16_t*>(p.side[side].grad) + at, d, 8);
  } else {
    __builtin_memcpy(static_cast<float*>(p.side[side].grad) + at, &v, 16);
  }
}

int32_t side_blocks(int64_t cols, int32_t rank) {
  return static_cast<int32_t>(((cols + 127) / 128 * ((rank + 15) / 16) + 3) / 4);
}

// Sizes and places of a backward call's workspace.
struct GradPlan {
  int64_t tiles, n_pad;
  int32_t splits[2], per_split[2];   // x, dy
  bool one_read;                     // of dy: dB and g together
  int64_t perm, adapter, tile0, bt, at, frag, part, g, h, wide, sums, outer, bytes;
  GradPlan(int64_t m, int64_t n, int64_t k, int32_t rank, int32_t n_adapters) {
    tiles = (m + kRowTile - 1) / kRowTile + (m < n_adapters ? m : n_adapters);   // at most
    if (tiles < 1) tiles = 1;
    n_pad = (n + 31) / 32 * 32;
    const int64_t chunks = (rank + 15) / 16;
    const int64_t jobs[2] = {(k + 127) / 128 * chunks, (n + 127) / 128 * chunks};
    // by adapter (per_split 0) while an adapter's tiles are few (4096 -> 4096,
    // rank 64: 1100 rows of 6 adapters 56 us, by range 67; of one 55 and 50;
    // 2051 of 24 adapters 97 and 118; 4096 rows of 6, 1001 columns 88 and 74)
    const bool by_adapter = m <= 512 * (n_adapters < 5 ? n_adapters : 5);
    // one read of a large dy (rank 16, one adapter: 8192 x 15360 136 us, two
    // reads 171; 2300 x 15360 59 and 63; 33000 x 1024 248 and 250; below 2^25
    // elements the second launch costs more, 16384 x 1024 149 and 139)
    one_read = !by_adapter && rank <= 16 && m * n >= (1 << 25);
    for (int side = 0; side < 2; ++side) {
      // as many waves as the chip holds at once, of at least four tiles, or
      // eight in a launch of its own (partial sums are written and read: 8192
      // rows of 15360 and 3840 columns 143 us with four, 136 with eight)
      int64_t want = kOuterWaves / (one_read ? jobs[side] : jobs[0] + jobs[1]);
      const int64_t most = tiles / (one_read ? 8 : 4);
      if (want > most) want = most;
      if (want < 1) want = 1;
      per_split[side] = by_adapter ? 0 : static_cast<int32_t>((tiles + want - 1) / want);
      splits[side] = by_adapter ? n_adapters
                                : static_cast<int32_t>((tiles + per_split[side] - 1) / per_split[side]);
    }
    bytes = 0;
    const auto place = [&](int64_t size) {
      const int64_t start = bytes;
      bytes += (size + 255) / 256 * 256;
      return start;
    };
    perm = place(tiles * kRowTile * 4);
    adapter = place(tiles * 4);
    tile0 = place((n_adapters + 1) * 4ll);
    bt = place(n_adapters * n_pad * rank * 2);
    at = place(n_adapters * k * rank * 2);
    frag = place(frag_bytes(m, rank));
    part = place(many_rows(m, k, n_adapters == 1) ? 0 : shrink_parts(m, n) * m * rank * 4);
    g = place(m * rank * 4);
    h = place(m * rank * 4);
    wide = place(n < 8 ? m * 16 : 0);
    sums = place(one_read ? side_blocks(n, rank) * tiles * kRowTile * 16 * 4 : 0);
    outer = place(by_adapter ? 0 : 2ll * rank * (splits[0] * k + splits[1] * n) * 4);
  }
  static constexpr int64_t kOuterWaves = 2048;
};

template <bool kSums>
void launch_outer(const OuterArgs& p, int64_t splits, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>(splits * (p.side[0].blocks + p.side[1].blocks)));
  if (p.o.perm != nullptr) hipLaunchKernelGGL((outer_kernel<kSums, true>), grid, dim3(256), 0, st, p);
  else hipLaunchKernelGGL((outer_kernel<kSums, false>), grid, dim3(256), 0, st, p);
}

// Row strides: 12 rows of fp32 stay below 2^31 bytes (32-bit lane offsets).
constexpr int64_t kMaxStride = 1 << 24;

bool sizes_ok(int64_t m, int64_t n, int64_t k, int32_t rank) {
  return m >= 0 && n >= 1 && k >= 1 && k % 32 == 0 && k <= (1 << 24) && n <= (1 << 24) &&
         m <= (1 << 24) && rank >= 8 && rank <= 128 && rank % 8 == 0;
}

int32_t check_common(const binade_lora* l, const uint16_t* x, int64_t m, int64_t ldx,
                     const void* workspace) {
  if (l == nullptr || m < 0 || l->n <= 0 || l->k <= 0 || l->rank <= 0 || l->n_adapters <= 0)
    return BINADE_EINVAL;
  if (!sizes_ok(m, l->n, l->k, l->rank) || l->n_adapters > 65535 || ldx > kMaxStride)
    return BINADE_EUNSUPPORTED;
  if (l->a == nullptr || l->b == nullptr) return BINADE_EINVAL;
  if (m > 0 && (x == nullptr || ldx < l->k)) return BINADE_EINVAL;
  if (!aligned16(l->a) || !aligned16(l->b) || !aligned16(x) || ldx % 8 != 0 ||
      !aligned16(workspace))
    return BINADE_EUNSUPPORTED;
  return BINADE_OK;
}

LoraArgs args_of(const binade_lora* l, int64_t m, const int32_t* ids, uint32_t* status) {
  return LoraArgs{l->a, l->b, l->scale, ids, l->n, l->k, m, l->rank, l->n_adapters, status};
}

}  // namespace
}  // namespace binade

using namespace binade;

extern "C" int64_t binade_lora_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t rank) {
  return sizes_ok(m, n, k, rank) ? add_workspace(m, n, k, rank) : 0;
}

extern "C" int64_t binade_lora_grad_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t rank,
                                                    int32_t n_adapters) {
  if (!sizes_ok(m, n, k, rank) || n_adapters < 1 || n_adapters > kMaxSorted) return 0;
  return GradPlan(m, n, k, rank, n_adapters).bytes;
}

extern "C" int32_t binade_lora_add(const binade_lora* l, const uint16_t* x, int64_t m, int64_t ldx,
                                   const int32_t* ids, const void* base, int64_t ld_base,
                                   int32_t base_dtype, void* y, int64_t ldy, int32_t y_dtype,
                                   float* h, void* workspace, int64_t workspace_bytes,
                                   uint32_t* dev_status, void* stream) {
  const int32_t s = check_common(l, x, m, ldx, workspace);
  if (s != BINADE_OK) return s;
  if ((base_dtype != BINADE_F32 && base_dtype != BINADE_BF16) ||
      (y_dtype != BINADE_F32 && y_dtype != BINADE_BF16))
    return BINADE_EINVAL;
  if (m == 0) return BINADE_OK;
  if (!aligned16(h)) return BINADE_EUNSUPPORTED;
  if (y == nullptr || ldy < l->n || (base != nullptr && ld_base < l->n)) return BINADE_EINVAL;
  if (ldy > kMaxStride || (base != nullptr && ld_base > kMaxStride)) return BINADE_EUNSUPPORTED;
  const int64_t need = binade_lora_workspace_bytes(m, l->n, l->k, l->rank);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return BINADE_ENOSPACE;
  const LoraArgs p = args_of(l, m, ids, dev_status);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const bool many = many_rows(m, p.n, ids == nullptr || p.n_adapters == 1);
  const int32_t parts = many ? 1 : shrink_parts(m, p.k);
  float* part = many ? nullptr : static_cast<float*>(workspace);
  uint4* frag = many ? static_cast<uint4*>(workspace) : nullptr;
  const ShrinkArgs sh{p, x, part, h, frag, ldx, p.k, slices_of(p.k), parts,
                      nullptr, nullptr, nullptr, (m + 15) / 16};
  const ExpandArgs ex{p, part, frag, base, y, h, ld_base, ldy, parts,
                      base == nullptr ? 0 : base_dtype == BINADE_BF16 ? 2 : 1,
                      y_dtype == BINADE_BF16, 0};
  if (one_pass(m, p.k, p.rank, p.n_adapters, ids != nullptr)) {
    if (p.rank <= 16) launch_one_ranks<1>(sh, ex, st);
    else launch_one_ranks<2>(sh, ex, st);
    return launch_status();
  }
  launch_shrink<false>(sh, st);
  launch_expand(ex, st);
  return launch_status();
}

extern "C" int32_t binade_lora_grad(const binade_lora* l, const uint16_t* x, int64_t m, int64_t ldx,
                                    const int32_t* ids, const uint16_t* dy, int64_t ld_dy,
                                    const float* h, const uint16_t* dx_base, int64_t ld_dx_base,
                                    uint16_t* dx, int64_t ld_dx, void* da, void* db,
                                    int32_t grad_dtype, void* workspace, int64_t workspace_bytes,
                                    uint32_t* dev_status, void* stream) {
  const int32_t s = check_common(l, x, m, ldx, workspace);
  if (s != BINADE_OK) return s;
  if (grad_dtype != BINADE_F32 && grad_dtype != BINADE_BF16) return BINADE_EINVAL;
  if (l->n_adapters > kMaxSorted) return BINADE_EUNSUPPORTED;
  if (da == nullptr || db == nullptr) return BINADE_EINVAL;
  if (m > 0 && (dy == nullptr || ld_dy < l->n)) return BINADE_EINVAL;
  if (ld_dy > kMaxStride) return BINADE_EUNSUPPORTED;
  if (!aligned16(da) || !aligned16(db) || !aligned16(h)) return BINADE_EUNSUPPORTED;
  if (dx != nullptr) {
    if (ld_dx < l->k || (dx_base != nullptr && ld_dx_base < l->k)) return BINADE_EINVAL;
    if (ld_dx > kMaxStride || (dx_base != nullptr && ld_dx_base > kMaxStride))
      return BINADE_EUNSUPPORTED;
    if (!aligned16(dx) || ld_dx % 8 != 0 ||
        (dx_base != nullptr && (!aligned16(dx_base) || ld_dx_base % 8 != 0)))
      return BINADE_EUNSUPPORTED;
  }
  if (m > 0 && (workspace == nullptr ||
                workspace_bytes <
                    binade_lora_grad_workspace_bytes(m, l->n, l->k, l->rank, l->n_adapters)))
    return BINADE_ENOSPACE;
  const LoraArgs p = args_of(l, m, ids, dev_status);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const GradPlan plan(m, p.n, p.k, p.rank, p.n_adapters);
  char* ws = static_cast<char*>(workspace);
  const auto floats = [&](int64_t at) { return reinterpret_cast<float*>(ws + at); };
  const auto ints = [&](int64_t at) { return reinterpret_cast<int32_t*>(ws + at); };
  const auto pieces = [&](int64_t at) { return reinterpret_cast<uint4*>(ws + at); };
  Order o{};
  o.tiles = static_cast<int32_t>((m + kRowTile - 1) / kRowTile);
  OuterArgs outer{};
  outer.scale = p.scale;
  outer.m = m;
  outer.rank = p.rank;
  outer.n_adapters = p.n_adapters;
  outer.grad_bf16 = grad_dtype == BINADE_BF16;
  if (m > 0 && p.n < 8) {
    uint16_t* wide = reinterpret_cast<uint16_t*>(ws + plan.wide);
    hipLaunchKernelGGL(widen_kernel, dim3(static_cast<uint32_t>((8 * m + 255) / 256)), dim3(256), 0,
                       st, dy, ld_dy, p.n, m, wide);
    dy = wide;
    ld_dy = 8;
  }
  outer.side[0] = OuterSide{x, nullptr, da, nullptr, ldx, p.k, p.k,
                            side_blocks(p.k, p.rank), plan.per_split[0]};
  outer.side[1] =
      OuterSide{dy, nullptr, db, nullptr, ld_dy, p.n, p.n < 8 ? 8 : p.n,
                side_blocks(p.n, p.rank), plan.per_split[1]};
  // without ids only adapter 0 is read
  const int32_t used = m == 0 ? 0 : ids != nullptr ? p.n_adapters : 1;
  uint16_t* bt = reinterpret_cast<uint16_t*>(ws + plan.bt);
  uint16_t* at = reinterpret_cast<uint16_t*>(ws + plan.at);
  PrepareArgs pre{};
  pre.p = p;
  pre.tb = TurnArgs{p.b, bt, p.n, p.rank, plan.n_pad, used};
  pre.ta = TurnArgs{p.a, at, p.rank, p.k, p.rank, dx != nullptr ? used : 0};
  if (m > 0 && ids != nullptr) {
    pre.perm = ints(plan.perm);
    pre.adapter = ints(plan.adapter);
    pre.tile0 = ints(plan.tile0);
    pre.sort_blocks = p.n_adapters;
    o.perm = pre.perm;
    o.adapter = pre.adapter;
    o.tile0 = pre.tile0;
  }
  pre.turns = (pre.tb.n_adapters * plan.n_pad + pre.ta.n_adapters * p.k) / 8 * (p.rank / 8);
  const int64_t turn_blocks = (pre.turns + 63) / 64;
  const uint32_t prepare_blocks =
      pre.sort_blocks + static_cast<uint32_t>(turn_blocks < (1 << 20) ? turn_blocks : 1 << 20);
  if (m > 0)
    hipLaunchKernelGGL(prepare_kernel, dim3(prepare_blocks), dim3(pre.sort_blocks > 0 ? 512 : 64), 0,
                       st, pre);
  if (m > 0) {
    if (h == nullptr) {
      launch_shrink<false>(ShrinkArgs{p, x, nullptr, floats(plan.h), pieces(plan.frag), ldx, p.k,
                                      slices_of(p.k), 1, nullptr, nullptr, nullptr, (m + 15) / 16},
                           st);
      h = floats(plan.h);
    }
    // g, and dx from it
    LoraArgs pg = p;
    pg.a = bt;
    pg.k = plan.n_pad;
    const bool whole =
        many_rows(m, p.k, ids == nullptr || p.n_adapters == 1) || dx == nullptr;
    const int32_t parts = whole || plan.one_read ? 1 : shrink_parts(m, p.n);
    float* const g = floats(plan.g);
    uint4* const frag = whole ? pieces(plan.frag) : nullptr;
    float* const part = plan.one_read ? g : floats(plan.part);
    outer.o = o;
    outer.side[0].v = g;
    outer.side[1].v = h;
    outer.side[0].part = floats(plan.outer);
    outer.side[1].part = floats(plan.outer) + 2ll * plan.splits[0] * p.rank * p.k;
    if (plan.one_read) {
      OuterArgs dy_alone = outer;
      dy_alone.side[0].blocks = 0;
      dy_alone.bt = bt;
      dy_alone.n_pad = plan.n_pad;
      dy_alone.sums = floats(plan.sums);
      dy_alone.tiles = plan.tiles;
      launch_outer<true>(dy_alone, plan.splits[1], st);
      hipLaunchKernelGGL(join_kernel, dim3(static_cast<uint32_t>((plan.tiles * 128 + 255) / 256)),
                         dim3(256), 0, st,
                         JoinArgs{p, o, dy_alone.sums, g, dx != nullptr ? frag : nullptr,
                                  plan.tiles, outer.side[1].blocks});
    } else {
      launch_shrink<true>(ShrinkArgs{pg, dy, whole ? nullptr : part, whole ? g : nullptr, frag,
                                     ld_dy, p.n, slices_of(p.n), parts, o.perm, o.adapter, o.tile0,
                                     o.perm != nullptr ? 2 * plan.tiles : (m + 15) / 16},
                          st);
    }
    if (dx != nullptr) {
      LoraArgs px = p;
      px.b = at;
      px.n = p.k;
      launch_expand(ExpandArgs{px, whole ? nullptr : part, frag, dx_base, dx,
                               whole || plan.one_read ? nullptr : g, ld_dx_base, ld_dx, parts,
                               dx_base == nullptr ? 0 : 2, true, 0},
                    st);
    }
  }
  OuterArgs rest = outer;
  if (plan.one_read) rest.side[1].blocks = 0;
  launch_outer<false>(rest, plan.splits[0], st);
  if (plan.per_split[0] > 0)
    hipLaunchKernelGGL(reduce_kernel,
                       dim3(static_cast<uint32_t>((p.rank * (p.n + p.k) / 4 + 255) / 256),
                            static_cast<uint32_t>(p.n_adapters)),
                       dim3(256), 0, st, outer);
  return launch_status();
}
