// Low-rank adapters beside a shared projection, forward and backward.
//
//   h[t] = A[i] x[t]              y[t] = base[t] + s[i] B[i] h[t]
//   g[t] = s[i] B[i]^T dy[t]      dx[t] = dx_base[t] + A[i]^T g[t]
//   dA[i] = sum_t g[t] x[t]^T     dB[i] = sum_t s[i] dy[t] h[t]^T
//
// for i = ids[t]. Plain form of each: one block per row for the rank-wide
// vectors, one thread per output for the rest.
#include <hip/hip_runtime.h>

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

constexpr int kSlice = 256;    // columns whose products one MFMA chain adds
constexpr int kStreams = 8;    // running sums the slices are dealt to

__device__ __forceinline__ bf16x8 as_bf16x8(uint4 v) { return __builtin_bit_cast(bf16x8, v); }

// 16 bytes at any 2-byte alignment (rows of an odd length).
__device__ __forceinline__ uint4 load8(const uint16_t* p) {
  uint4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// Two fp32 values rounded to bf16, nearest-even, packed (gfx950 converts).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float float2v __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((float2v{a, b}), bf16x2));
}

// v = hi + mid + lo exactly, each a bf16 (8 significant bits by truncation):
// fp32 values enter a bf16 MFMA as three terms and lose nothing. Infinity
// and NaN stay in hi alone.
__device__ __forceinline__ void split3(float v, uint16_t& hi, uint16_t& mid, uint16_t& lo) {
  const uint32_t u = __float_as_uint(v), top = u & 0xFFFF0000u;
  float rest = v - __uint_as_float(top);
  if ((u & 0x7F800000u) == 0x7F800000u) rest = 0.0f;
  const uint32_t m = __float_as_uint(rest) & 0xFFFF0000u;
  hi = static_cast<uint16_t>(top >> 16);
  mid = static_cast<uint16_t>(m >> 16);
  lo = static_cast<uint16_t>(__float_as_uint(rest - __uint_as_float(m)) >> 16);
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
struct ShrinkArgs {
  LoraArgs p;
  const uint16_t* x;
  float* out;
  int64_t ldx;
  int32_t slices, parts;   // parts: 1 (whole), 8 (streams) or slices
};

template <int RT>
__global__ __launch_bounds__(512) void shrink_kernel(ShrinkArgs s) {
  const LoraArgs& p = s.p;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int64_t row = row0 + i < p.m ? row0 + i : p.m - 1;
  const int32_t id = row0 + i < p.m ? adapter_of(p, row) : -1;
  if (blockIdx.y == 0 && threadIdx.x < 16 && p.status != nullptr && p.ids != nullptr && id < 0 &&
      row0 + i < p.m && p.ids[row] != -1)
    atomicOr(p.status, static_cast<uint32_t>(BINADE_DEV_BAD_INDEX));
  const int32_t first = s.parts == 1 ? wave : static_cast<int32_t>(blockIdx.y);
  const int32_t step = s.parts <= kStreams ? kStreams : s.slices;
  int32_t idq[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) idq[q] = __shfl(id, 4 * g + q, 64);
  floatx4 mine[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) mine[r] = floatx4{0, 0, 0, 0};
  const uint16_t* xr = s.x + row * s.ldx + 8 * g;
  uint32_t todo = static_cast<uint32_t>(__ballot(id >= 0)) & 0xFFFFu;
  uint32_t got = wave == 0 ? 0xFFFFu & ~todo : 0u;   // rows whose sums this wave holds
  for (int32_t turn = 0; todo != 0; ++turn) {
    const int32_t a = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    const uint32_t match = static_cast<uint32_t>(__ballot(id == a)) & 0xFFFFu;
    todo &= ~match;
    if (s.parts > 1 && turn % static_cast<int32_t>(blockDim.x >> 6) != wave) continue;
    got |= match;
    const uint16_t* ar[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int32_t rr = 16 * r + i < p.rank ? 16 * r + i : p.rank - 1;
      ar[r] = p.a + (static_cast<int64_t>(a) * p.rank + rr) * p.k + 8 * g;
    }
    floatx4 sum[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) sum[r] = floatx4{0, 0, 0, 0};
    for (int32_t c = first; c < s.slices; c += step) {
      const int64_t col = static_cast<int64_t>(c) * kSlice;
      floatx4 acc[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r] = floatx4{0, 0, 0, 0};
      if (p.k - col >= kSlice) {
        uint4 xf[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) xf[j] = *reinterpret_cast<const uint4*>(xr + col + 32 * j);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          uint4 af[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) af[j] = *reinterpret_cast<const uint4*>(ar[r] + col + 32 * j);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(xf[j]), as_bf16x8(af[j]),
                                                             acc[r], 0, 0, 0);
        }
      } else {
        for (int64_t cc = col; cc < p.k; cc += 32) {
          const uint4 xf = *reinterpret_cast<const uint4*>(xr + cc);
#pragma unroll
          for (int r = 0; r < RT; ++r)
            acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                as_bf16x8(xf), as_bf16x8(*reinterpret_cast<const uint4*>(ar[r] + cc)), acc[r], 0, 0,
                0);
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) sum[r] += acc[r];
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (idq[q] == a) mine[r][q] = sum[r][q];
  }
  if (s.parts > 1) {
    float* out = s.out + static_cast<int64_t>(blockIdx.y) * p.m * p.rank;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t t = row0 + 4 * g + q;
        if (t < p.m && 16 * r + i < p.rank && (got >> (4 * g + q)) & 1u)
          out[t * p.rank + 16 * r + i] = mine[r][q];
      }
    return;
  }
  __shared__ float sums[kStreams][16][16 * RT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int q = 0; q < 4; ++q) sums[wave][4 * g + q][16 * r + i] = mine[r][q];
  __syncthreads();
  const int32_t live = s.slices < kStreams ? s.slices : kStreams;
  for (int32_t e = threadIdx.x; e < 16 * p.rank; e += 512) {
    const int32_t t = e / p.rank, r = e - t * p.rank;
    float v = 0.0f;
    for (int32_t w = 0; w < live; ++w) v += sums[w][t][r];
    if (row0 + t < p.m) s.out[(row0 + t) * p.rank + r] = v;
  }
}

// y[t] = base[t] + s[i] B[i] h[t]: 16 MT rows by 64 CT columns a block of
// four waves, each wave 16 CT columns. h is split into three bf16 terms in
// LDS; B's rows go straight into MFMA operands and stay in registers for the
// block's row tiles of one adapter. Column c of a wave's MFMA tiles is spread
// so that lane i ends with the CT adjacent columns CT i .. CT i + CT - 1. A
// tile of 16 rows runs once for each adapter among them; base is loaded one
// tile ahead of its use.
struct ExpandArgs {
  LoraArgs p;
  const float* part;
  const void* base;
  void* y;
  float* h;
  int64_t ld_base, ldy;
  int32_t parts;           // of the first product: 1, 8 or its slices
  int32_t base_kind;       // 0 none, 1 fp32, 2 bf16
  bool y_bf16;
};

// The sum of a value's partial sums in the order of the first product, four
// ranks at a time: at is the first of parts partials, next apart.
template <int kAhead>
__device__ __forceinline__ floatx4 join_parts(const float* at, int64_t next, int32_t parts) {
  floatx4 v{0, 0, 0, 0};
  if (parts == 1) return *reinterpret_cast<const floatx4*>(at);
  floatx4 sum[kStreams];
#pragma unroll
  for (int w = 0; w < kStreams; ++w) sum[w] = floatx4{0, 0, 0, 0};
  for (int32_t c = 0; c < parts; c += kAhead * kStreams) {
    floatx4 d[kAhead][kStreams];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int w = 0; w < kStreams; ++w) {
        const int32_t q = c + j * kStreams + w;
        d[j][w] = floatx4{0, 0, 0, 0};
        if (q < parts) d[j][w] = *reinterpret_cast<const floatx4*>(at + q * next);
      }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int w = 0; w < kStreams; ++w) sum[w] += d[j][w];
  }
#pragma unroll
  for (int w = 0; w < kStreams; ++w) v += sum[w];
  return v;
}

// Kinds of base and y.
constexpr int kNone = 0, kF32 = 1, kBf16 = 2;

template <int CT, int BK>
struct BaseTile {
  uint32_t d[4][BK == kNone ? 1 : BK == kBf16 ? CT / 2 : CT];   // four rows' values, as loaded
};

template <int KS, int MT, int CT, int BK, int YK>
__global__ __launch_bounds__(256) void expand_kernel(ExpandArgs s) {
  const LoraArgs& p = s.p;
  constexpr int kRows = 16 * MT, kLd = 32 * KS + 8;
  __shared__ __align__(16) uint16_t hs[3][kRows][kLd];
  __shared__ __align__(16) int32_t ids[kRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * kRows;
  const int32_t rows = static_cast<int32_t>(p.m - row0 < kRows ? p.m - row0 : kRows);
  const int64_t col = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * (16 * CT) + CT * i;
  const bool full = col + CT <= p.n;

  BaseTile<CT, BK> ahead;
  auto load_base = [&](int m) {
    if (BK == kNone || !full) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = 16 * m + 4 * g + q;
      const int64_t at = (row0 + (t < rows ? t : rows - 1)) * s.ld_base + col;
      if (BK == kBf16)
        __builtin_memcpy(ahead.d[q], static_cast<const uint16_t*>(s.base) + at, 2 * CT);
      else
        __builtin_memcpy(ahead.d[q], static_cast<const float*>(s.base) + at, 4 * CT);
    }
  };
  if (threadIdx.x < kRows)
    ids[threadIdx.x] =
        static_cast<int32_t>(threadIdx.x) < rows ? adapter_of(p, row0 + threadIdx.x) : -2;
  load_base(0);
  for (int32_t e = threadIdx.x; e < kRows * 8 * KS; e += 256) {
    const int32_t t = e / (8 * KS), r = 4 * (e % (8 * KS));
    floatx4 v{0, 0, 0, 0};
    if (r < p.rank && t < rows) {
      const int64_t at = (row0 + t) * p.rank + r;
      v = join_parts<MT == 1 ? 4 : 1>(s.part + at, p.m * p.rank, s.parts);
      if (s.h != nullptr && blockIdx.x == 0) *reinterpret_cast<floatx4*>(s.h + at) = v;
    }
    uint16_t d[3][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) split3(v[j], d[0][j], d[1][j], d[2][j]);
#pragma unroll
    for (int part = 0; part < 3; ++part) __builtin_memcpy(&hs[part][t][r], d[part], 8);
  }
  __syncthreads();

  uint4 bf[CT][KS];
  int32_t loaded = -1;
  float scale = 1.0f;
#pragma unroll 1
  for (int m = 0; 16 * m < rows; ++m) {
    const BaseTile<CT, BK> base = ahead;
    if (16 * (m + 1) < rows) load_base(m + 1);
    int32_t idq[4];
    __builtin_memcpy(idq, &ids[16 * m + 4 * g], 16);
    const int32_t id = ids[16 * m + i];
    floatx4 mine[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) mine[c] = floatx4{0, 0, 0, 0};
    uint64_t todo = __ballot(id >= 0) & 0xFFFFu;
    while (todo != 0) {
      const int32_t a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
      todo &= ~__ballot(id == a);
      if (a != loaded) {
        loaded = a;
        scale = p.scale != nullptr ? p.scale[a] : 1.0f;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const int64_t n = col + c < p.n ? col + c : p.n - 1;
          const uint16_t* b = p.b + (static_cast<int64_t>(a) * p.n + n) * p.rank;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const int32_t o = 32 * k + 8 * g;
            bf[c][k] = *reinterpret_cast<const uint4*>(b + (o < p.rank ? o : 0));
          }
        }
        // ranks beyond the last: zeros (h has zeros there too)
#pragma unroll
        for (int k = 0; k < KS; ++k)
          if (32 * k + 32 > p.rank) {
            const bool live = 32 * k + 8 * g < p.rank;
#pragma unroll
            for (int c = 0; c < CT; ++c) {
              bf[c][k].x = live ? bf[c][k].x : 0u;
              bf[c][k].y = live ? bf[c][k].y : 0u;
              bf[c][k].z = live ? bf[c][k].z : 0u;
              bf[c][k].w = live ? bf[c][k].w : 0u;
            }
          }
      }
      floatx4 acc[CT];
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[c] = floatx4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const bf16x8 hf = as_bf16x8(
              *reinterpret_cast<const uint4*>(&hs[part][16 * m + i][32 * k + 8 * g]));
#pragma unroll
          for (int c = 0; c < CT; ++c)
            acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hf, as_bf16x8(bf[c][k]), acc[c], 0, 0,
                                                             0);
        }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool hit = idq[q] == a;
#pragma unroll
        for (int c = 0; c < CT; ++c) mine[c][q] = hit ? scale * acc[c][q] : mine[c][q];
      }
    }
    if (full) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int t = 16 * m + 4 * g + q;
        float f[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          float b = 0.0f;
          if (BK == kBf16)
            b = c & 1 ? bf16_hi(base.d[q][c / 2]) : bf16_lo(base.d[q][c / 2]);
          else if (BK == kF32)
            b = __uint_as_float(base.d[q][c]);
          f[c] = idq[q] < 0 ? b : b + mine[c][q];
        }
        if (t >= rows) continue;
        const int64_t at = (row0 + t) * s.ldy + col;
        if (YK == kBf16) {
          uint32_t d[CT / 2];
#pragma unroll
          for (int c = 0; c < CT / 2; ++c) d[c] = pack_bf16(f[2 * c], f[2 * c + 1]);
          __builtin_memcpy(static_cast<uint16_t*>(s.y) + at, d, 2 * CT);
        } else {
          __builtin_memcpy(static_cast<float*>(s.y) + at, f, 4 * CT);
        }
      }
    } else if (col < p.n) {   // the row's last columns, one by one
#pragma unroll
      for (int c = 0; c < CT - 1; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int t = 16 * m + 4 * g + q;
          if (t >= rows || col + c >= p.n) continue;
          const float b = BK == kNone ? 0.0f
                                      : load_any(s.base, (row0 + t) * s.ld_base + col + c,
                                                 BK == kBf16);
          store_any(s.y, (row0 + t) * s.ldy + col + c, YK == kBf16,
                    idq[q] < 0 ? b : b + mine[c][q]);
        }
    }
  }
}

int32_t slices_of(int64_t k) { return static_cast<int32_t>((k + kSlice - 1) / kSlice); }

// Whether the second product's blocks of 64 rows by 512 columns fill the
// chip; blocks of 16 by 128 otherwise.
bool wide_expand(int64_t m, int64_t n) {
  return ((m + 63) / 64) * ((n + 511) / 512) >= 256;
}

// Grain of the first product: partial sums it leaves per value.
int32_t shrink_parts(int64_t m, int64_t n, int64_t k) {
  const int64_t tiles = (m + 15) / 16;
  const int32_t slices = slices_of(k);
  if (tiles >= 128 || slices == 1) return 1;
  if ((tiles * kStreams >= 256 || wide_expand(m, n)) && slices > kStreams) return kStreams;
  return slices;
}

void launch_shrink(const LoraArgs& p, const uint16_t* x, int64_t ldx, int32_t parts, float* out,
                   hipStream_t st) {
  const ShrinkArgs s{p, x, out, ldx, slices_of(p.k), parts};
  const dim3 grid(static_cast<uint32_t>((p.m + 15) / 16), parts == 1 ? 1u : static_cast<uint32_t>(parts));
  const int64_t mixed = p.ids == nullptr || p.m < p.n_adapters ? p.m : p.n_adapters;
  const dim3 block(parts == 1 ? 64 * kStreams
                   : p.ids == nullptr || mixed < 2 ? 64
                   : mixed < 8 ? 256 : 512);
  if (p.rank <= 16) hipLaunchKernelGGL(shrink_kernel<1>, grid, block, 0, st, s);
  else if (p.rank <= 32) hipLaunchKernelGGL(shrink_kernel<2>, grid, block, 0, st, s);
  else if (p.rank <= 64) hipLaunchKernelGGL(shrink_kernel<4>, grid, block, 0, st, s);
  else hipLaunchKernelGGL(shrink_kernel<8>, grid, block, 0, st, s);
}

template <int KS, int BK, int YK>
void launch_expand_shape(const ExpandArgs& s, hipStream_t st) {
  const int64_t m = s.p.m, n = s.p.n;
  const auto grid = [&](int64_t rows, int64_t cols) {
    return dim3(static_cast<uint32_t>((n + cols - 1) / cols),
                static_cast<uint32_t>((m + rows - 1) / rows));
  };
  if (wide_expand(m, n))
    hipLaunchKernelGGL((expand_kernel<KS, 4, 8, BK, YK>), grid(64, 512), dim3(256), 0, st, s);
  else
    hipLaunchKernelGGL((expand_kernel<KS, 1, 2, BK, YK>), grid(16, 128), dim3(256), 0, st, s);
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
  else launch_expand_ranks<4>(s, st);
}

// --------------------------------------------------------------- backward
// out[t, r] = scale * sum over c of v[t, c] * w[c, r], w strided (A by rows
// of r, B by rows of c); one block per row, one wave per rank in turn.
__global__ __launch_bounds__(256) void rows_kernel(LoraArgs p, const uint16_t* v, int64_t ldv,
                                                   const uint16_t* w, int64_t cols,
                                                   int64_t stride_r, int64_t stride_c, bool scaled,
                                                   float* out) {
  const int64_t t = blockIdx.x;
  const int32_t i = adapter_of(p, t);
  if (threadIdx.x == 0 && i < 0 && p.status != nullptr && p.ids[t] != -1)
    atomicOr(p.status, static_cast<uint32_t>(BINADE_DEV_BAD_INDEX));
  const int lane = threadIdx.x & 63;
  const uint16_t* wi = w + static_cast<int64_t>(i < 0 ? 0 : i) * p.rank * cols;
  for (int32_t r = threadIdx.x >> 6; r < p.rank; r += 4) {
    float acc = 0.0f;
    if (i >= 0)
      for (int64_t c = lane; c < cols; c += 64)
        acc = __builtin_fmaf(bf16_f32(v[t * ldv + c]), bf16_f32(wi[r * stride_r + c * stride_c]),
                             acc);
    acc = slot_tree(acc);
    if (lane == 0) {
      if (scaled && i >= 0 && p.scale != nullptr) acc *= p.scale[i];
      out[t * p.rank + r] = acc;
    }
  }
}

// out[t, c] = base[t, c] + scale * sum over r of v[t, r] * w[c, r].
__global__ __launch_bounds__(256) void add_kernel(LoraArgs p, const float* v, const uint16_t* w,
                                                     int64_t cols, int64_t stride_r,
                                                     int64_t stride_c, bool scaled,
                                                     const void* base, int64_t ld_base,
                                                     bool base_bf16, void* out, int64_t ld_out,
                                                     bool out_bf16) {
  const int64_t total = p.m * cols;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < total;
       e += step) {
    const int64_t t = e / cols, c = e - t * cols;
    const int32_t i = adapter_of(p, t);
    float y = base != nullptr ? load_any(base, t * ld_base + c, base_bf16) : 0.0f;
    if (i >= 0) {
      const uint16_t* wi = w + static_cast<int64_t>(i) * p.rank * cols;
      float acc = 0.0f;
      for (int32_t r = 0; r < p.rank; ++r)
        acc = __builtin_fmaf(v[t * p.rank + r], bf16_f32(wi[r * stride_r + c * stride_c]), acc);
      if (scaled && p.scale != nullptr) acc *= p.scale[i];
      y = y + acc;
    }
    store_any(out, t * ld_out + c, out_bf16, y);
  }
}

// grad[i, r, c] = scale * sum over rows t of adapter i of v[t, r] * s[t, c].
__global__ __launch_bounds__(256) void outer_kernel(LoraArgs p, const float* v, const uint16_t* s,
                                                    int64_t lds, int64_t cols, int64_t stride_r,
                                                    int64_t stride_c, bool scaled, void* grad,
                                                    bool grad_bf16) {
  const int64_t per = static_cast<int64_t>(p.rank) * cols;
  const int64_t total = per * p.n_adapters;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < total;
       e += step) {
    const int32_t i = static_cast<int32_t>(e / per);
    const int64_t at = e - i * per, r = at / cols, c = at - r * cols;
    double acc = 0.0;
    for (int64_t t = 0; t < p.m; ++t)
      if (adapter_of(p, t) == i)
        acc += static_cast<double>(v[t * p.rank + r]) * static_cast<double>(bf16_f32(s[t * lds + c]));
    if (scaled && p.scale != nullptr) acc *= p.scale[i];
    store_any(grad, i * per + r * stride_r + c * stride_c, grad_bf16, static_cast<float>(acc));
  }
}

uint32_t blocks_for(int64_t n) {
  const int64_t b = (n + 255) / 256;
  return static_cast<uint32_t>(b < 65536 ? b : 65536);
}

bool sizes_ok(int64_t m, int64_t n, int64_t k, int32_t rank) {
  return m >= 0 && n >= 1 && k >= 1 && k % 32 == 0 && k <= (1 << 30) && n <= (1 << 30) &&
         m <= (1 << 30) && rank >= 8 && rank <= 128 && rank % 8 == 0;
}

int32_t check_common(const binade_lora* l, const uint16_t* x, int64_t m, int64_t ldx,
                     const void* workspace) {
  if (l == nullptr || m < 0 || l->n <= 0 || l->k <= 0 || l->rank <= 0 || l->n_adapters <= 0)
    return BINADE_EINVAL;
  if (!sizes_ok(m, l->n, l->k, l->rank) || l->n_adapters > 65535) return BINADE_EUNSUPPORTED;
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
  return sizes_ok(m, n, k, rank) ? shrink_parts(m, n, k) * m * rank * 4 : 0;
}

extern "C" int64_t binade_lora_grad_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t rank,
                                                    int32_t n_adapters) {
  return sizes_ok(m, n, k, rank) && n_adapters >= 1 && n_adapters <= 65535 ? 2 * m * rank * 4 : 0;
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
  if (y == nullptr || ldy < l->n || (base != nullptr && ld_base < l->n)) return BINADE_EINVAL;
  if (workspace_bytes < binade_lora_workspace_bytes(m, l->n, l->k, l->rank) ||
      workspace == nullptr)
    return BINADE_ENOSPACE;
  const LoraArgs p = args_of(l, m, ids, dev_status);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int32_t parts = shrink_parts(m, p.n, p.k);
  float* part = parts == 1 && h != nullptr ? h : static_cast<float*>(workspace);
  launch_shrink(p, x, ldx, parts, part, st);
  launch_expand(ExpandArgs{p, part, base, y, h, ld_base, ldy, parts,
                           base == nullptr ? 0 : base_dtype == BINADE_BF16 ? 2 : 1,
                           y_dtype == BINADE_BF16},
                st);
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
  if (da == nullptr || db == nullptr) return BINADE_EINVAL;
  if (m > 0 && (dy == nullptr || ld_dy < l->n)) return BINADE_EINVAL;
  if (dx != nullptr) {
    if (ld_dx < l->k || (dx_base != nullptr && ld_dx_base < l->k)) return BINADE_EINVAL;
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
  const bool gb = grad_dtype == BINADE_BF16;
  float* g = static_cast<float*>(workspace);
  float* hw = g + m * p.rank;
  if (m > 0) {
    hipLaunchKernelGGL(rows_kernel, dim3(static_cast<uint32_t>(m)), dim3(256), 0, st, p, dy, ld_dy,
                       p.b, p.n, static_cast<int64_t>(1), static_cast<int64_t>(p.rank), true, g);
    if (h == nullptr) {
      hipLaunchKernelGGL(rows_kernel, dim3(static_cast<uint32_t>(m)), dim3(256), 0, st, p, x, ldx,
                         p.a, p.k, p.k, static_cast<int64_t>(1), false, hw);
      h = hw;
    }
    if (dx != nullptr)
      hipLaunchKernelGGL(add_kernel, dim3(blocks_for(m * p.k)), dim3(256), 0, st, p, g, p.a, p.k,
                         p.k, static_cast<int64_t>(1), false, static_cast<const void*>(dx_base),
                         ld_dx_base, true, static_cast<void*>(dx), ld_dx, true);
  }
  hipLaunchKernelGGL(outer_kernel, dim3(blocks_for(p.n_adapters * p.rank * p.k)), dim3(256), 0, st,
                     p, g, x, ldx, p.k, p.k, static_cast<int64_t>(1), false, da, gb);
  hipLaunchKernelGGL(outer_kernel, dim3(blocks_for(p.n_adapters * p.rank * p.n)), dim3(256), 0, st,
                     p, h, dy, ld_dy, p.n, static_cast<int64_t>(1), static_cast<int64_t>(p.rank),
                     true, db, gb);
  return launch_status();
}
