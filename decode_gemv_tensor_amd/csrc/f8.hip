// Matrix products in 8-bit floating point with a scale for each block of 128
// (the arithmetic is stated in binade.h): of a projection, its gradients, and
// of the experts that a router chose.
//
// A block's scale is a power of two for everything that is quantised here, so
// that v 2^-e is exact and the only rounding is the one to e4m3. Weights of a
// checkpoint may come with any fp32 scale for 128 x 128 values: then each
// block's 128 columns are summed from zero and added with one fma.
//
// The operands (e4m3 times a power of two is exact in bf16) go through
// v_mfma_f32_16x16x32_bf16, whose products are exact and whose sums are fp32's.
// The instructions on 8-bit operands are not used: they add eight products
// after cutting them to 13 bits below the largest (1.4e-5 of the result's norm
// for normal data, 5e-5 for values spread over the whole range, where this one
// has 1e-8 and 8e-8; up to 2% of the results round to another bf16). The one
// of 16x16x128 would run at twice the rate (4.3 against 2.3 PFLOP/s), the one
// of 16x16x32, which cuts alike, at the same.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "binade.h"
#include "device_common.h"

namespace binade {
namespace {

using namespace dev;

typedef int int8v __attribute__((ext_vector_type(8)));
typedef int int4v __attribute__((ext_vector_type(4)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short short2v __attribute__((ext_vector_type(2)));
typedef unsigned short ushort2v __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int64_t kMaxSize = 1 << 22;    // of m, n and k: a tile's offsets fit 32 bits
constexpr int64_t kMaxPairs = 1 << 24;   // (token, slot) pairs of an expert product
constexpr int kMaxExperts = 4096;        // of an expert product
constexpr int kSmallRows = 16;           // rows of one few-row pass
constexpr int kSmallPairs = 256;         // pairs that the few-row kernel sorts by itself

__host__ __device__ inline int64_t blocks_of(int64_t n) { return (n + 127) / 128; }
inline int64_t padded(int64_t n) { return blocks_of(n) * 128; }
inline int64_t codes_of(int64_t n) { return (blocks_of(n) + 3) / 4 * 4; }   // bytes of a row's codes
inline int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

// ------------------------------------------------------------------- scales
// The code (exponent + 127) of a block whose largest finite |v| has the bf16
// bits u: the least e >= -126 with |v| <= 448 2^e = 1.75 2^(e+8).
__device__ __forceinline__ uint32_t code_of(uint32_t u) {
  const int32_t c = static_cast<int32_t>(u >> 7) - 8 + ((u & 127u) > 96u ? 1 : 0);
  return u == 0 ? 127u : c < 1 ? 1u : static_cast<uint32_t>(c);
}
__device__ __forceinline__ float scale_of_code(uint32_t c) { return __uint_as_float(c << 23); }
// The same for a code that a checkpoint brought: 0 is 2^-127, 255 NaN.
__device__ __forceinline__ float scale_of_any_code(uint32_t c) {
  return __uint_as_float(c == 0 ? 0x00400000u : c == 255u ? 0x7FC00000u : c << 23);
}

// Larger magnitude of two pairs of bf16 bits; infinities and NaN count as 0.
__device__ __forceinline__ uint32_t finite_abs(uint32_t v) {
  const uint32_t a = v & 0x7FFF7FFFu;
  const uint32_t lo = (a & 0xFFFFu) >= 0x7F80u ? 0u : a & 0xFFFFu;
  return a >= 0x7F800000u ? lo : lo | (a & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(ushort2v, a),
                                                               __builtin_bit_cast(ushort2v, b)));
}
__device__ __forceinline__ uint32_t max_of_pair(uint32_t a) {
  const uint32_t lo = a & 0xFFFFu, hi = a >> 16;
  return lo > hi ? lo : hi;
}

// Four bf16 (two dwords) as four e4m3 bytes of v / s: to the nearest, ties to
// even; infinities and NaN become NaN.
__device__ __forceinline__ uint32_t to_f8(uint32_t a, uint32_t b, float s) {
  short2v o = {0, 0};
  o = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, __builtin_bit_cast(bf16x2, a), s, false);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, __builtin_bit_cast(bf16x2, b), s, true);
  return __builtin_bit_cast(uint32_t, o);
}
// Eight e4m3 bytes as bf16, times s (a power of two: exact).
__device__ __forceinline__ bf16x8 from_f8(uint32_t a, uint32_t b, float s) {
  const bf16x2 p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, false);
  const bf16x2 q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, true);
  const bf16x2 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, false);
  const bf16x2 t = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, true);
  return bf16x8{p[0], p[1], q[0], q[1], r[0], r[1], t[0], t[1]};
}

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(v), kCtrl, 0xF, 0xF, true));
}
// The largest of 16 neighbouring lanes, in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  uint32_t o = dpp<0xB1>(v);   // quad_perm 1 0 3 2
  v = o > v ? o : v;
  o = dpp<0x4E>(v);            // quad_perm 2 3 0 1
  v = o > v ? o : v;
  o = dpp<0x141>(v);           // row_half_mirror
  v = o > v ? o : v;
  o = dpp<0x140>(v);           // row_mirror
  return o > v ? o : v;
}
// The largest of the lanes l, l^16, l^32, l^48.
__device__ __forceinline__ uint32_t max_rows(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = a[0] > a[1] ? a[0] : a[1];
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return b[0] > b[1] ? b[0] : b[1];
}

// Eight bf16 of a row from column c on (zeros behind the last of n).
__device__ __forceinline__ void load8(const uint16_t* row, int64_t c, int64_t n, bool vec,
                                      uint32_t (&d)[4]) {
  if (vec) {   // n is a multiple of 8 and rows are 16-byte aligned
    uint4 v{0, 0, 0, 0};
    if (c < n) v = *reinterpret_cast<const uint4*>(row + c);
    d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = c + 2 * j < n ? row[c + 2 * j] : 0u;
      const uint32_t hi = c + 2 * j + 1 < n ? row[c + 2 * j + 1] : 0u;
      d[j] = lo | (hi << 16);
    }
  }
}

// ----------------------------------------------------------------- quantise
// Operands lie block by block of 128 columns, a block's rows one behind the
// other: a tile's step is one piece of memory, whatever the row's length (rows
// of 15360 bytes one below the other meet only four of an L2's sixteen
// channels: 1.5 times the time of a large product).
//
// Rows of v [m, n] as e4m3, blocks_of(n) blocks of m_pad rows, with a code
// for each block of a row: 16 lanes a block, 8 values a lane.
__device__ __forceinline__ void quantise_rows(const uint16_t* v, int64_t ld, int64_t m, int64_t n,
                                              bool vec, uint8_t* q, int64_t m_pad, uint8_t* codes,
                                              int64_t ldc, int64_t first, int64_t step) {
  const int64_t nb = blocks_of(n), units = m * nb;
  const int l = threadIdx.x & 15;
#pragma unroll 2
  for (int64_t u = first; u < units; u += step) {
    const int64_t row = u / nb, b = u - row * nb;
    uint32_t d[4];
    load8(v + row * ld, b * 128 + l * 8, n, vec, d);
    const uint32_t top = max16(max_of_pair(max_pair(max_pair(finite_abs(d[0]), finite_abs(d[1])),
                                                    max_pair(finite_abs(d[2]), finite_abs(d[3])))));
    const uint32_t code = code_of(top);
    const float s = scale_of_code(code);
    *reinterpret_cast<uint2*>(q + (b * m_pad + row) * 128 + l * 8) =
        uint2{to_f8(d[0], d[1], s), to_f8(d[2], d[3], s)};
    if (l == 0) codes[row * ldc + b] = static_cast<uint8_t>(code);
  }
}

__global__ __launch_bounds__(256) void quantise_rows_kernel(const uint16_t* v, int64_t ld,
                                                            int64_t m, int64_t n, bool vec,
                                                            uint8_t* q, int64_t m_pad, uint8_t* codes,
                                                            int64_t ldc) {
  quantise_rows(v, ld, m, n, vec, q, m_pad, codes, ldc,
                static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4),
                static_cast<int64_t>(gridDim.x) * 16);
}

// 128 x 128 tiles of v [m, n], turned: qt of n_pad rows with codes for 128
// rows of a column, and (kRows) also as quantise_rows_kernel leaves them; or
// (kOne) with one code for the tile, as weights are kept, q and (qt not NULL)
// qt. A tile lies in LDS as pairs of columns; rows 32 apart, which four
// neighbouring lanes read at once, are 16 banks apart.
struct TileArgs {
  const uint16_t* v;
  int64_t ld, m, n;
  uint8_t *q, *codes, *qt, *codes_t;
  int64_t m_pad, n_pad;      // rows of a block of q, of qt
  int64_t ldc, ldct;
  int64_t v_next, q_next, c_next, qt_next, ct_next;   // from one matrix to the next
  bool vec;
};

constexpr int kPitch = 66;
__device__ __forceinline__ int tile_at(int row, int pair) {
  return row * kPitch + (row >> 5) * 16 + pair;
}

template <bool kRows, bool kOne>
__global__ __launch_bounds__(256) void quantise_tile_kernel(TileArgs p) {
  __shared__ uint32_t tile[128 * kPitch + 64];
  __shared__ uint32_t tops[4];
  const int t = threadIdx.x, l = t & 15;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 128, c0 = static_cast<int64_t>(blockIdx.x) * 128;
  const uint16_t* v = p.v + blockIdx.z * p.v_next;
  uint32_t d[8][4], top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = r0 + i * 16 + (t >> 4);
    if (row < p.m) load8(v + row * p.ld, c0 + l * 8, p.n, p.vec, d[i]);
    else d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0;
  }
  uint32_t code = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = max_pair(max_pair(finite_abs(d[i][0]), finite_abs(d[i][1])),
                                max_pair(finite_abs(d[i][2]), finite_abs(d[i][3])));
    if (kOne) top = max_pair(top, a);
    const int row = i * 16 + (t >> 4);
    if (kRows) {
      const uint32_t c = code_of(max16(max_of_pair(a)));
      const float s = scale_of_code(c);
      if (r0 + row < p.m) {
        *reinterpret_cast<uint2*>(p.q + (blockIdx.x * p.m_pad + r0 + row) * 128 + l * 8) =
            uint2{to_f8(d[i][0], d[i][1], s), to_f8(d[i][2], d[i][3], s)};
        if (l == 0) p.codes[(r0 + row) * p.ldc + blockIdx.x] = static_cast<uint8_t>(c);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) tile[tile_at(row, l * 4 + j)] = d[i][j];
  }
  if (kOne) {
    top = max_rows(max16(max_of_pair(top)));
    if ((t & 63) == 0) tops[t >> 6] = top;
  }
  __syncthreads();
  if (kOne) {
    top = tops[0];
#pragma unroll
    for (int w = 1; w < 4; ++w) top = tops[w] > top ? tops[w] : top;
    code = code_of(top);
    const float s = scale_of_code(code);
    uint8_t* q = p.q + blockIdx.z * p.q_next;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = r0 + i * 16 + (t >> 4);
      if (row < p.m)
        *reinterpret_cast<uint2*>(q + (blockIdx.x * p.m_pad + row) * 128 + l * 8) =
            uint2{to_f8(d[i][0], d[i][1], s), to_f8(d[i][2], d[i][3], s)};
    }
    if (t == 0) {
      p.codes[blockIdx.z * p.c_next + blockIdx.y * p.ldc + blockIdx.x] = static_cast<uint8_t>(code);
      if (p.qt != nullptr)
        p.codes_t[blockIdx.z * p.ct_next + blockIdx.x * p.ldct + blockIdx.y] =
            static_cast<uint8_t>(code);
    }
    if (p.qt == nullptr) return;
  }
  // a lane: 32 rows (quarter t & 3) of two columns
  const int quarter = t & 3, pair = t >> 2;
  uint32_t c[32], a = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    c[i] = tile[tile_at(quarter * 32 + i, pair)];
    if (!kOne) a = max_pair(a, finite_abs(c[i]));
  }
  uint32_t code_lo = code, code_hi = code;
  if (!kOne) {
    a = max_pair(a, dpp<0xB1>(a));
    a = max_pair(a, dpp<0x4E>(a));
    code_lo = code_of(a & 0xFFFFu);
    code_hi = code_of(a >> 16);
  }
  uint8_t* qt = p.qt + blockIdx.z * p.qt_next;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t col = c0 + pair * 2 + h;
    if (col >= p.n) continue;
    const uint32_t cc = h ? code_hi : code_lo;
    const float s = scale_of_code(cc);
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      constexpr uint32_t kLo = 0x05040100u, kHi = 0x07060302u;
      o[i] = to_f8(vperm(c[4 * i + 1], c[4 * i], h ? kHi : kLo),
                   vperm(c[4 * i + 3], c[4 * i + 2], h ? kHi : kLo), s);
    }
    uint4* out = reinterpret_cast<uint4*>(qt + (blockIdx.y * p.n_pad + col) * 128 + quarter * 32);
    out[0] = uint4{o[0], o[1], o[2], o[3]};
    out[1] = uint4{o[4], o[5], o[6], o[7]};
    if (!kOne && quarter == 0)
      p.codes_t[col * p.ldct + blockIdx.y] = static_cast<uint8_t>(cc);
  }
}

// ------------------------------------------------------------------- layout
// e4m3 bytes [rows, cols] into blocks of 128 columns, zeros behind, and turned.
struct LayoutArgs {
  const uint8_t* v;
  uint8_t *q, *qt;
  int64_t rows, cols;
};

__global__ __launch_bounds__(256) void layout_kernel(LayoutArgs p) {
  __shared__ uint32_t tile[128][33];
  const int t = threadIdx.x;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 128, c0 = static_cast<int64_t>(blockIdx.x) * 128;
  const uint8_t* v = p.v + blockIdx.z * p.rows * p.cols;
  const int64_t z = blockIdx.z;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = i * 32 + (t >> 3), piece = t & 7;
    const int64_t c = c0 + piece * 16;
    uint4 d{0, 0, 0, 0};
    if (r0 + row < p.rows && c < p.cols)   // cols is a multiple of 16
      d = *reinterpret_cast<const uint4*>(v + (r0 + row) * p.cols + c);
    if (r0 + row < p.rows)
      *reinterpret_cast<uint4*>(p.q + ((z * gridDim.x + blockIdx.x) * p.rows + r0 + row) * 128 +
                                piece * 16) = d;
    tile[row][piece * 4] = d.x;
    tile[row][piece * 4 + 1] = d.y;
    tile[row][piece * 4 + 2] = d.z;
    tile[row][piece * 4 + 3] = d.w;
  }
  if (p.qt == nullptr) return;
  __syncthreads();
  // a lane: four columns (a dword) of 16 rows
  const int four = t >> 3, part = t & 7;
  uint32_t o[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = tile[part * 16 + 4 * i][four], b = tile[part * 16 + 4 * i + 1][four];
    const uint32_t c = tile[part * 16 + 4 * i + 2][four], d = tile[part * 16 + 4 * i + 3][four];
    const uint32_t ab0 = vperm(b, a, 0x05010400u), cd0 = vperm(d, c, 0x05010400u);
    const uint32_t ab1 = vperm(b, a, 0x07030602u), cd1 = vperm(d, c, 0x07030602u);
    o[0][i] = vperm(cd0, ab0, 0x05040100u);
    o[1][i] = vperm(cd0, ab0, 0x07060302u);
    o[2][i] = vperm(cd1, ab1, 0x05040100u);
    o[3][i] = vperm(cd1, ab1, 0x07060302u);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t col = c0 + four * 4 + j;
    if (col < p.cols)
      *reinterpret_cast<uint4*>(p.qt + ((z * gridDim.y + blockIdx.y) * p.cols + col) * 128 + part * 16) =
          uint4{o[j][0], o[j][1], o[j][2], o[j][3]};
  }
}

// Scales [count, nb, kb] into rows of a multiple of four, and turned.
template <typename T>
__global__ __launch_bounds__(256) void layout_scales_kernel(const T* s, T* out, T* out_t,
                                                            int64_t count, int64_t nb, int64_t kb) {
  const int64_t total = count * nb * kb, kb4 = (kb + 3) / 4 * 4, nb4 = (nb + 3) / 4 * 4;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t k = i % kb, r = i / kb, n = r % nb, z = r / nb;
    if (out != nullptr) out[(z * nb + n) * kb4 + k] = s[i];
    if (out_t != nullptr) out_t[(z * kb + k) * nb4 + n] = s[i];
  }
}

// ------------------------------------------------------------------ product
// Scales of the weights' side: a code for 128 x 128 values, a code for 128
// columns of each row, or an fp32 number for 128 x 128 values.
enum Scales { kBlockCode, kRowCode, kBlockF32 };

struct GemmArgs {
  const uint8_t *x, *x_codes, *w;
  const void* w_scales;
  void* y;
  float* part;             // [splits, m, n], or NULL: one split, straight to y
  int64_t x_block, w_block;   // bytes of a block of 128 columns
  int64_t ldy, m, n;
  int32_t ld_xc, ld_ws;    // codes or scales of a row
  int32_t kb, per_split, splits, mt, nt;
  bool y_bf16, y_vec;
  // experts: pairs by expert, tiles of them, and a matrix's size
  const int32_t* order;
  const int4* tiles;       // expert (-1: none, -2: no tile), first pair, pairs
  int64_t w_next, s_next;
  int32_t pairs_a_row;
};

// Blocks go to the eight XCDs in turn: number them so that an XCD has a
// connected range, and take the range in columns of eight row tiles, so that
// the tiles at work at once on an XCD share their rows in its L2.
__device__ __forceinline__ bool tile_of(const GemmArgs& p, int32_t& mt, int32_t& nt, int32_t& split) {
  const int32_t total = gridDim.x, per = total / 8, more = total % 8;
  const int32_t xcd = blockIdx.x % 8, local = blockIdx.x / 8;
  int32_t id = xcd * per + (xcd < more ? xcd : more) + local;
  const int32_t tiles = p.mt * p.nt;
  split = id / tiles;
  id -= split * tiles;
  constexpr int32_t kGroup = 8;
  const int32_t group = id / (kGroup * p.nt), first = group * kGroup;
  const int32_t high = p.mt - first < kGroup ? p.mt - first : kGroup;
  id -= group * kGroup * p.nt;
  mt = first + id % high;
  nt = id / high;
  return split < p.splits;
}

__device__ __forceinline__ void to_lds(const uint8_t* from, uint8_t* to) {
  __builtin_amdgcn_global_load_lds(from, (lds_void*)to, 16, 0, 0);
}

// Four results of a row, from column col on.
__device__ __forceinline__ void store4(const GemmArgs& p, int32_t split, int64_t row, int64_t col,
                                       floatx4 v) {
  if (p.part != nullptr) {
    float* to = p.part + (split * p.m + row) * p.n + col;
    if (p.n % 4 == 0) {
      if (col < p.n) *reinterpret_cast<floatx4*>(to) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < p.n) to[e] = v[e];
    }
    return;
  }
  const int64_t at = row * p.ldy + col;
  if (p.y_vec) {   // rows of whole, aligned fours of fp32
    if (col < p.n) *reinterpret_cast<floatx4*>(static_cast<float*>(p.y) + at) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (col + e >= p.n) continue;
      if (p.y_bf16) static_cast<uint16_t*>(p.y)[at + e] = to_bf16_rne(v[e]);
      else static_cast<float*>(p.y)[at + e] = v[e];
    }
  }
}

// Experts' tiles: an XCD's share of the places (p.mt), in columns of eight.
__device__ __forceinline__ void expert_tile_of(const GemmArgs& p, int32_t& mt, int32_t& nt) {
  const int32_t xcd = blockIdx.x % 8, local = blockIdx.x / 8;
  constexpr int32_t kGroup = 8;
  const int32_t group = local / (kGroup * p.nt), first = group * kGroup;
  const int32_t high = p.mt - first < kGroup ? p.mt - first : kGroup;
  const int32_t at = local - group * kGroup * p.nt;
  mt = xcd * p.mt + first + at % high;
  nt = at / high;
}

// y = x w^T on tiles of BM x BN by WM x WN waves. A step is one block of 128
// columns: its BM + BN rows of 128 bytes go straight to LDS, one step ahead of
// their use, into two buffers (named arrays: the compiler then sees that reads
// of one do not wait for loads of the other). In LDS a row's eight 16-byte
// pieces are swizzled by row / 2, so that the 16 rows of an operand read touch
// every bank once; the swizzle is in the addresses that the lanes load from.
// The weights are the instruction's first operand: a lane's four results lie
// side by side in a row of y.
// Every variant is held to two waves a SIMD (256 registers): the few that took
// more by themselves lost more from waiting alone than from what they spill
// (2048 x 4096 x 4096 with fp32 results and scales 101 -> 85 us, experts of
// 4096 x 8 pairs alike 358 -> 256 us; with powers of two 74 -> 72, 229 -> 231).
// Bound by vector instructions beside the matrix ones: both operands become
// bf16 here, two conversions for each matrix instruction of a wave's 64 x 64,
// 3.7 instructions with everything. Two are hidden behind a matrix instruction
// (7.2 ns a slot of a SIMD with one, 7.8 with two, 11.4 with four). 4096 x
// 15360 x 3840: 390 us, 1.24 PFLOP/s; 15360 x 3840 x 8192 (a weight's gradient)
// 0.83 to 0.95 ms, 1.02 to 1.16; a large bf16 library product has 1.6 (tiles of
// 256 rows, a wave's 128 or 64 of them: 1.13 and 0.97 ms). With experts and few
// blocks of K the ends of the tiles count too: runs of two to six tiles a
// block, the next one's loads under way over an end, spill and gain nothing.
template <int BM, int BN, int WM, int WN, int kScales, bool kExperts>
__global__ __launch_bounds__(64 * WM * WN, 2) void gemm_kernel(GemmArgs p) {
  constexpr int kWaves = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr int kXLoads = BM / 8 / kWaves, kWLoads = BN / 8 / kWaves;
  static_assert(kXLoads * 8 * kWaves == BM && kWLoads * 8 * kWaves == BN, "whole loads");
  static_assert(TN <= 128 && 128 % TN == 0, "a wave's columns have one scale");
  __shared__ __align__(16) uint8_t buf0[(BM + BN) * 128];
  __shared__ __align__(16) uint8_t buf1[(BM + BN) * 128];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4, wm = wave / WN, wn = wave % WN;
  int32_t mt, nt, split;
  if (kExperts) {
    expert_tile_of(p, mt, nt);
    split = blockIdx.y;   // 0
  } else if (!tile_of(p, mt, nt, split)) {
    return;
  }
  const int64_t n0 = static_cast<int64_t>(nt) * BN;
  int64_t m0 = static_cast<int64_t>(mt) * BM, rows = p.m - m0;
  const uint8_t* w = p.w;
  int64_t expert = 0;
  if (kExperts) {
    const int4 tile = p.tiles[mt];
    if (tile.x == -2) return;
    expert = tile.x;
    m0 = tile.y;
    rows = tile.z;
    w += (expert < 0 ? 0 : expert) * p.w_next;
  }
  const int32_t kb0 = split * p.per_split;
  const int32_t kb1 = kb0 + p.per_split < p.kb ? kb0 + p.per_split : p.kb;

  // where this lane's 16-byte pieces come from
  const int piece_row = lane >> 3;
  const auto piece = [&](int row) { return ((lane & 7) ^ ((row >> 1) & 7)) * 16; };
  int64_t x_off[kExperts ? kXLoads : 1];
  uint32_t w_off[kWLoads];
  const uint8_t* x = p.x + (kExperts ? 0 : m0 * 128);
#pragma unroll
  for (int i = 0; i < (kExperts ? kXLoads : 1); ++i) {
    const int row = (i * kWaves + wave) * 8 + piece_row;
    const int32_t pair = kExperts ? p.order[m0 + (row < rows ? row : 0)] : 0;
    x_off[i] = (kExperts ? static_cast<int64_t>(pair / p.pairs_a_row) : row) * 128 + piece(row);
  }
  w += n0 * 128;
#pragma unroll
  for (int i = 0; i < kWLoads; ++i) {
    const int row = (i * kWaves + wave) * 8 + piece_row;
    const int64_t at = n0 + row < p.n ? row : p.n - 1 - n0;
    w_off[i] = static_cast<uint32_t>(at * 128 + piece(row));
  }
  const auto stage = [&](uint8_t* buf, int32_t kb) __attribute__((always_inline)) {
    const uint8_t* xk = x + kb * p.x_block;
    const uint8_t* wk = w + kb * p.w_block;
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)   // 32 rows or more on, the pieces lie the same way
      to_lds(kExperts ? xk + x_off[kExperts ? i : 0]
                      : xk + (i * kWaves * 1024 + static_cast<uint64_t>(static_cast<uint32_t>(x_off[0]))),
             buf + (i * kWaves + wave) * 1024);
#pragma unroll
    for (int i = 0; i < kWLoads; ++i)
      to_lds(wk + static_cast<uint64_t>(w_off[i]), buf + BM * 128 + (i * kWaves + wave) * 1024);
  };

  // codes of four steps at once: of the rows of x, and of the weights
  uint32_t xc_off[FM], wc_off[kScales == kRowCode ? FN : 1];
  int64_t xc_base = 0;
  if (!kExperts) xc_base = m0 * p.ld_xc;
  const uint8_t* x_codes = p.x_codes + xc_base;
  int64_t xc_row[kExperts ? FM : 1];
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int row = wm * TM + i * 16 + r;
    if (kExperts) {
      const int32_t pair = p.order[m0 + (row < rows ? row : 0)];
      xc_row[kExperts ? i : 0] = static_cast<int64_t>(pair / p.pairs_a_row) * p.ld_xc;
    } else {
      xc_off[i] = static_cast<uint32_t>(row * p.ld_xc);
    }
  }
  const uint8_t* w_codes = static_cast<const uint8_t*>(p.w_scales);
  const float* w_f32 = static_cast<const float*>(p.w_scales);
  if (kScales == kRowCode) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int64_t row = n0 + wn * TN + j * 16 + r;
      wc_off[j] = static_cast<uint32_t>((row < p.n ? row : p.n - 1) - n0) * p.ld_ws;
    }
    w_codes += n0 * p.ld_ws;
  } else {
    const int64_t first = n0 + uniform(wn * TN);
    const int64_t at = (expert < 0 ? 0 : expert) * p.s_next + (first < p.n ? first : p.n - 1) / 128 * p.ld_ws;
    w_codes += at;
    w_f32 += at;
  }
  uint32_t xc[FM], xc_next[FM], wc[kScales == kRowCode ? FN : 1], wc_next[kScales == kRowCode ? FN : 1];
  float wf[4], wf_next[4];
  const auto request = [&](int32_t kb) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
      xc_next[i] = kExperts
          ? *reinterpret_cast<const uint32_t*>(x_codes + xc_row[kExperts ? i : 0] + kb)
          : *reinterpret_cast<const uint32_t*>(x_codes + kb + static_cast<uint64_t>(xc_off[i]));
    if (kScales == kRowCode) {
#pragma unroll
      for (int j = 0; j < (kScales == kRowCode ? FN : 1); ++j)
        wc_next[j] = *reinterpret_cast<const uint32_t*>(w_codes + kb + static_cast<uint64_t>(wc_off[j]));
    } else if (kScales == kBlockCode) {
      wc_next[0] = *reinterpret_cast<const uint32_t*>(w_codes + kb);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) wf_next[j] = w_f32[kb + j];
    }
  };

  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  const uint32_t at0 = r * 128 + ((q ^ ((r >> 1) & 7)) << 4), at1 = at0 ^ 64;
  const auto operand = [&](const uint8_t* rows16) __attribute__((always_inline)) {
    const int4v a = *reinterpret_cast<const int4v*>(rows16 + at0);
    const int4v b = *reinterpret_cast<const int4v*>(rows16 + at1);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  const auto compute = [&](const uint8_t* buf, auto step) __attribute__((always_inline)) {
    constexpr int kStep = decltype(step)::value;
    const uint8_t* xb = buf + wm * TM * 128;
    const uint8_t* wb = buf + (BM + wn * TN) * 128;
    bf16x8 wv[FN][4];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int8v v = operand(wb + j * 2048);
      const uint32_t c = kScales == kBlockF32 ? 127u : (wc[kScales == kRowCode ? j : 0] >> (8 * kStep)) & 255u;
      const float s = kScales == kBlockCode ? scale_of_any_code(c) : scale_of_code(c);
#pragma unroll
      for (int h = 0; h < 4; ++h) wv[j][h] = from_f8(v[2 * h], v[2 * h + 1], s);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int8v v = operand(xb + i * 2048);
      const float s = scale_of_code((xc[i] >> (8 * kStep)) & 255u);
      bf16x8 xv[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) xv[h] = from_f8(v[2 * h], v[2 * h + 1], s);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        floatx4 sum = kScales == kBlockF32 ? floatx4{0.0f, 0.0f, 0.0f, 0.0f} : acc[i][j];
#pragma unroll
        for (int h = 0; h < 4; ++h)
          sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j][h], xv[h], sum, 0, 0, 0);
        if (kScales == kBlockF32) {
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(wf[kStep], sum[e], acc[i][j][e]);
        } else {
          acc[i][j] = sum;
        }
      }
    }
  };
  // The loads into LDS are waited for by hand (the compiler does not count
  // them before a barrier).
  const auto arrived = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    __syncthreads();
  };

  if (kb0 < kb1 && expert >= 0) {
    request(kb0);
    stage(buf0, kb0);
    for (int32_t kb = kb0; kb < kb1; kb += 4) {
      const auto one = [&](auto step, uint8_t* cur, uint8_t* other) __attribute__((always_inline)) {
        constexpr int kStep = decltype(step)::value;
        if (kb + kStep >= kb1) return;
        arrived();
        if (kStep == 0) {
#pragma unroll
          for (int i = 0; i < FM; ++i) xc[i] = xc_next[i];
#pragma unroll
          for (int j = 0; j < (kScales == kRowCode ? FN : 1); ++j) wc[j] = wc_next[j];
#pragma unroll
          for (int j = 0; j < 4; ++j) wf[j] = wf_next[j];
          if (kb + 4 < kb1) request(kb + 4);
        }
        if (kb + kStep + 1 < kb1) stage(other, kb + kStep + 1);
        compute(cur, step);
      };
      one(std::integral_constant<int, 0>(), buf0, buf1);
      one(std::integral_constant<int, 1>(), buf1, buf0);
      one(std::integral_constant<int, 2>(), buf0, buf1);
      one(std::integral_constant<int, 3>(), buf1, buf0);
    }
  }

  // a lane: rows i * 16 + r, columns j * 16 + 4 q .. + 3
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int row = wm * TM + i * 16 + r;
    const bool live = row < rows;
    const int64_t y_row = kExperts ? static_cast<int64_t>(p.order[m0 + (live ? row : 0)]) : m0 + row;
    const int64_t col0 = n0 + wn * TN;
    if (p.part == nullptr && p.y_bf16 && p.y_vec) {
      // the halves of two operands' results change places between lanes 16
      // apart: eight columns a lane, 64 bytes of a row side by side
#pragma unroll
      for (int j = 0; j < FN; j += 2) {
        const floatx4 a = acc[i][j], b = acc[i][j + 1];
        const auto lo = __builtin_amdgcn_permlane16_swap(pack_bf16(a[0], a[1]), pack_bf16(b[0], b[1]), false,
                                                         false);
        const auto hi = __builtin_amdgcn_permlane16_swap(pack_bf16(a[2], a[3]), pack_bf16(b[2], b[3]), false,
                                                         false);
        const int64_t col = col0 + (j + (q & 1)) * 16 + (q & 2) * 4;
        if (live && col < p.n)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y) + y_row * p.ldy + col) =
              uint4{lo[0], hi[0], lo[1], hi[1]};
      }
    } else if (live) {
#pragma unroll
      for (int j = 0; j < FN; ++j) store4(p, split, y_row, col0 + j * 16 + q * 4, acc[i][j]);
    }
  }
}

// The splits' sums, in their order. Only outputs of up to 128 tiles are
// split: m * n fits 32 bits. 8 splits of 61 x 3840: 3.0 us, the launch itself.
template <int kEach>
__global__ __launch_bounds__(256) void join_kernel(const float* part, int32_t splits, uint32_t total,
                                                   uint32_t n, void* y, int64_t ldy, bool y_bf16) {
  typedef float values __attribute__((ext_vector_type(kEach)));
  for (uint32_t i = (blockIdx.x * 256 + threadIdx.x) * kEach; i < total; i += gridDim.x * 256 * kEach) {
    values s = *reinterpret_cast<const values*>(part + i);
#pragma unroll 4
    for (int32_t k = 1; k < splits; ++k)
      s += *reinterpret_cast<const values*>(part + static_cast<int64_t>(k) * total + i);
    const uint32_t row = i / n;
    const int64_t at = row * ldy + (i - row * n);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      if (y_bf16) static_cast<uint16_t*>(y)[at + e] = to_bf16_rne(s[e]);
      else static_cast<float*>(y)[at + e] = s[e];
    }
  }
}

__global__ __launch_bounds__(256) void zero_kernel(uint32_t* p, int64_t words) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < words;
       i += static_cast<int64_t>(gridDim.x) * 256)
    p[i] = 0;
}

// ------------------------------------------------------------ few-row product
// Up to 16 rows of x at a time: the weights are read once (15360 x 3840, one
// row: 16.6 us a pass with weights in the cache, 18.2 with ten matrices in turn,
// 59 MB; 64 pairs of 55 of 128 experts, 704 x 2816: 26.6, and 29.0 from memory,
// 109 MB). Bound by vector instructions more than by that: 6.9 million for the
// row, 13 us on 1024 SIMDs at 2.1 GHz; of a step's 239 the weights' conversions
// are 16, most others find the largest of x and quantise it in each wave. A block
// has 16 NR rows of w; its waves take blocks of 128 columns in turn, weights
// and rows of x straight into the operands' registers (lane: row l % 16,
// columns 16 q .. and 64 + 16 q ..; x in the same order), x quantised there.
// With experts, a block is one pair's: the first pair of an expert does all
// of that expert's pairs, the others' blocks end at once.
struct SmallArgs {
  const uint16_t* x;
  const uint8_t* w;
  const void* w_scales;
  void* y;
  int64_t ldx, ldy, n, k;
  int32_t m, ld_ws;
  bool y_bf16;
  const int32_t* idx;     // experts
  uint32_t* status;
  int64_t w_next, s_next;
  int32_t n_experts, pairs_a_row;
};

template <int NR, int kWaves, int kScales, bool kExperts>
__global__ __launch_bounds__(64 * kWaves) void few_rows_kernel(SmallArgs p) {
  __shared__ float red[kWaves][NR * 16][17];
  __shared__ int32_t pairs[kExperts ? kSmallPairs : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * NR);
  int32_t m = p.m, expert = 0;
  if (kExperts) {
    const int32_t mine = blockIdx.y;
    expert = p.idx[mine];
    if (expert < 0 || expert >= p.n_experts) {
      if (expert != -1 && blockIdx.x == 0 && threadIdx.x == 0 && p.status != nullptr)
        atomicOr(p.status, static_cast<uint32_t>(BINADE_DEV_BAD_INDEX));
      for (int i = threadIdx.x; i < 16 * NR; i += 64 * kWaves) {
        if (n0 + i >= p.n) break;
        const int64_t at = mine * p.ldy + n0 + i;
        if (p.y_bf16) static_cast<uint16_t*>(p.y)[at] = 0;
        else static_cast<float*>(p.y)[at] = 0.0f;
      }
      return;
    }
    // every wave for itself: the pairs of this expert, in order
    m = 0;
    for (int32_t i0 = 0; i0 < p.m; i0 += 64) {
      const bool same = i0 + lane < p.m && p.idx[i0 + lane] == expert;
      const uint64_t hits = __ballot(same);
      if (m == 0 && hits != 0 && i0 + __builtin_ctzll(hits) < mine) return;
      if (wave == 0 && same) pairs[m + __popcll(hits & ((1ull << lane) - 1))] = i0 + lane;
      m += __popcll(hits);
    }
    __syncthreads();
  }
  const int32_t kb = static_cast<int32_t>((p.k + 127) / 128);
  const uint8_t* w = p.w + expert * p.w_next;
  const uint8_t* w_row[NR];
  int64_t s_row[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int64_t row = n0 + i * 16 + r;
    w_row[i] = w + (row < p.n ? row : p.n - 1) * 128 + q * 16;
    const int64_t first = n0 + i * 16 < p.n ? n0 + i * 16 : p.n - 1;
    s_row[i] = expert * p.s_next + first / 128 * p.ld_ws;
  }
  for (int32_t m0 = 0; m0 < m; m0 += kSmallRows) {
    const bool live = m0 + r < m;
    const int32_t pair = kExperts ? pairs[live ? m0 + r : 0] : (live ? m0 + r : 0);
    const uint16_t* x = p.x + static_cast<int64_t>(kExperts ? pair / p.pairs_a_row : pair) * p.ldx;
    floatx4 acc[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) acc[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    uint4 wn[NR][2], xn[4];
    const auto request = [&](int32_t b) __attribute__((always_inline)) {
      const int64_t k = static_cast<int64_t>(b) * 128;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        wn[i][0] = *reinterpret_cast<const uint4*>(w_row[i] + b * p.n * 128);
        wn[i][1] = *reinterpret_cast<const uint4*>(w_row[i] + b * p.n * 128 + 64);
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int64_t c = k + (h >> 1) * 64 + q * 16 + (h & 1) * 8;
        xn[h] = uint4{0, 0, 0, 0};
        if (live && c < p.k) xn[h] = *reinterpret_cast<const uint4*>(x + c);
      }
    };
    if (wave < kb) request(wave);
    for (int32_t b = wave; b < kb; b += kWaves) {
      uint4 wv[NR][2];
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        wv[i][0] = wn[i][0];
        wv[i][1] = wn[i][1];
      }
      uint32_t d[16];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        d[4 * h] = xn[h].x;
        d[4 * h + 1] = xn[h].y;
        d[4 * h + 2] = xn[h].z;
        d[4 * h + 3] = xn[h].w;
      }
      if (b + kWaves < kb) request(b + kWaves);
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) top = max_pair(top, d[j] & 0x7FFF7FFFu);
      if (__ballot((top & 0xFFFFu) >= 0x7F80u || top >= 0x7F800000u) != 0) {   // rare
        top = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) top = max_pair(top, finite_abs(d[j]));
      }
      const float s = scale_of_code(code_of(max_rows(max_of_pair(top))));
      bf16x8 xv[4];
#pragma unroll
      for (int h = 0; h < 4; ++h)
        xv[h] = from_f8(to_f8(d[4 * h], d[4 * h + 1], s), to_f8(d[4 * h + 2], d[4 * h + 3], s), s);
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float ws = 1.0f;
        if (kScales == kBlockCode)
          ws = scale_of_any_code(static_cast<const uint8_t*>(p.w_scales)[s_row[i] + b]);
        floatx4 sum = kScales == kBlockF32 ? floatx4{0.0f, 0.0f, 0.0f, 0.0f} : acc[i];
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(from_f8(wv[i][0].x, wv[i][0].y, ws), xv[0], sum, 0, 0, 0);
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(from_f8(wv[i][0].z, wv[i][0].w, ws), xv[1], sum, 0, 0, 0);
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(from_f8(wv[i][1].x, wv[i][1].y, ws), xv[2], sum, 0, 0, 0);
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(from_f8(wv[i][1].z, wv[i][1].w, ws), xv[3], sum, 0, 0, 0);
        if (kScales == kBlockF32) {
          ws = static_cast<const float*>(p.w_scales)[s_row[i] + b];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] = __builtin_fmaf(ws, sum[e], acc[i][e]);
        } else {
          acc[i] = sum;
        }
      }
    }
    // lane: column r of x's rows, w rows 4 q .. + 3
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][i * 16 + q * 4 + e][r] = acc[i][e];
    __syncthreads();
    for (int o = threadIdx.x; o < NR * 256; o += 64 * kWaves) {
      const int n = o % (NR * 16), row = o / (NR * 16);
      if (m0 + row >= m || n0 + n >= p.n) continue;
      float s = red[0][n][row];
#pragma unroll
      for (int v = 1; v < kWaves; ++v) s += red[v][n][row];
      const int64_t at = static_cast<int64_t>(kExperts ? pairs[m0 + row] : m0 + row) * p.ldy + n0 + n;
      if (p.y_bf16) static_cast<uint16_t*>(p.y)[at] = to_bf16_rne(s);
      else static_cast<float*>(p.y)[at] = s;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ pairs by expert
// One block: counts, the tiles of each expert's pairs, and the pairs in their
// experts' order, those without expert last (within one expert in whatever
// order: a row's result does not depend on its place). The other blocks
// quantise the rows meanwhile. Tiles lie as the product's blocks take them: an
// eighth for each XCD, with its share of the tiles that have an expert,
// connected, then its share of the others (expert -1: zeros), then none (-2).
// (With tiles numbered through, the last XCDs have few that are in use.)
// 32768 pairs take 27 us, a chain of loads, LDS atomics and sums over experts
// of one block, beside the rows' quantising (72 MB, 14 us at a copy's rate).
struct SortArgs {
  const int32_t* idx;
  int32_t pairs, n_experts, bm, share;   // share: places of tiles of an XCD
  int32_t* order;
  int4* tiles;
  uint32_t* status;
};

// Eight ids of a thread, thread by thread: an expert, n_experts for none, -1
// behind the last pair.
__device__ __forceinline__ bool ids_of(const SortArgs& p, int32_t from, int32_t (&e)[8]) {
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int32_t i = from + j * 1024;
    e[j] = i < p.pairs ? p.idx[i] : INT32_MIN;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool none = e[j] < 0 || e[j] >= p.n_experts, in = from + j * 1024 < p.pairs;
    bad |= in && none && e[j] != -1;
    e[j] = !in ? -1 : none ? p.n_experts : e[j];
  }
  return bad;
}

// Counts eight ids a lane. Pairs without expert are many where tokens are
// padded: one addition a wave for them.
__device__ __forceinline__ void count_behind(int32_t* cursor, const int32_t (&e)[8], int32_t none, int lane) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint64_t nones = __ballot(e[j] == none);
    if (e[j] == none ? (nones & ((1ull << lane) - 1)) == 0 : e[j] >= 0)
      atomicAdd(&cursor[e[j]], e[j] == none ? __popcll(nones) : 1);
  }
}
// And gives each its place.
__device__ __forceinline__ void place_behind(int32_t* cursor, const int32_t (&e)[8], int32_t none, int lane,
                                             int32_t (&at)[8]) {
  uint64_t nones[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    nones[j] = __ballot(e[j] == none);
    at[j] = 0;
    if (e[j] == none ? (nones[j] & ((1ull << lane) - 1)) == 0 : e[j] >= 0)
      at[j] = atomicAdd(&cursor[e[j]], e[j] == none ? __popcll(nones[j]) : 1);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int32_t first = __shfl(at[j], nones[j] != 0 ? __builtin_ctzll(nones[j]) : 0, 64);
    if (e[j] == none) at[j] = first + __popcll(nones[j] & ((1ull << lane) - 1));
  }
}

__device__ void sort_pairs(const SortArgs& p) {
  __shared__ int32_t cursor[kMaxExperts + 1], first_tile[kMaxExperts + 1];
  __shared__ int32_t sums[2][16];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const bool few = p.pairs <= 32768;   // then ids stay in registers
  int32_t held[4][8];
  bool bad = false;
  if (few) {
#pragma unroll
    for (int b = 0; b < 4; ++b) bad |= ids_of(p, t + b * 8192, held[b]);
  }
  for (int32_t e = t; e <= p.n_experts; e += 1024) cursor[e] = 0;
  for (int32_t i = t; i < 8 * p.share; i += 1024) p.tiles[i] = int4{-2, 0, 0, 0};
  __syncthreads();
  if (few) {
#pragma unroll
    for (int b = 0; b < 4; ++b) count_behind(cursor, held[b], p.n_experts, lane);
  } else {
    for (int32_t from = t; from - t < p.pairs; from += 8192) {
      int32_t e[8];
      bad |= ids_of(p, from, e);
      count_behind(cursor, e, p.n_experts, lane);
    }
  }
  if (bad && p.status != nullptr) atomicOr(p.status, static_cast<uint32_t>(BINADE_DEV_BAD_INDEX));
  __syncthreads();
  // starts: sums over the experts before, 1024 at a time. A start replaces the
  // count; the next start, or the pairs' number, ends it.
  int32_t pair_base = 0, tile_base = 0;
  for (int32_t e0 = 0; e0 <= p.n_experts; e0 += 1024) {
    const int32_t e = e0 + t;
    const int32_t n = e <= p.n_experts ? cursor[e] : 0, k = (n + p.bm - 1) / p.bm;
    int32_t ps = n, ts = k;
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t a = __shfl_up(ps, d, 64), b = __shfl_up(ts, d, 64);
      if (lane >= d) {
        ps += a;
        ts += b;
      }
    }
    if (lane == 63) {
      sums[0][wave] = ps;
      sums[1][wave] = ts;
    }
    __syncthreads();
    int32_t before_p = pair_base, before_t = tile_base;
    for (int v = 0; v < 16; ++v) {
      if (v < wave) {
        before_p += sums[0][v];
        before_t += sums[1][v];
      }
      pair_base += sums[0][v];
      tile_base += sums[1][v];
    }
    if (e <= p.n_experts) {
      cursor[e] = before_p + ps - n;
      first_tile[e] = before_t + ts - k;
    }
    __syncthreads();
  }
  const int32_t live = first_tile[p.n_experts], per = live / 8, more = live % 8;
  for (int32_t e = t; e <= p.n_experts; e += 1024) {
    const int32_t start = cursor[e], end = e < p.n_experts ? cursor[e + 1] : p.pairs;
    for (int32_t j = 0; start + j * p.bm < end; ++j) {
      const int32_t i = first_tile[e] + j;
      int32_t xcd, place;
      if (e < p.n_experts) {
        const int32_t larger = more * (per + 1);   // tiles of the XCDs with one more
        xcd = i < larger ? i / (per + 1) : more + (i - larger) / per;
        place = i < larger ? i % (per + 1) : (i - larger) % per;
      } else {
        xcd = j % 8;
        place = per + (xcd < more ? 1 : 0) + j / 8;
      }
      p.tiles[xcd * p.share + place] =
          int4{e < p.n_experts ? e : -1, start + j * p.bm,
               end - start - j * p.bm < p.bm ? end - start - j * p.bm : p.bm, 0};
    }
  }
  __syncthreads();   // starts are read above and moved on below
  if (few) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      int32_t to[8];
      place_behind(cursor, held[b], p.n_experts, lane, to);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (held[b][j] >= 0) p.order[to[j]] = t + b * 8192 + j * 1024;
    }
    return;
  }
  for (int32_t from = t; from - t < p.pairs; from += 8192) {
    int32_t e[8], to[8];
    ids_of(p, from, e);
    place_behind(cursor, e, p.n_experts, lane, to);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e[j] >= 0) p.order[to[j]] = from + j * 1024;
  }
}

__global__ __launch_bounds__(1024) void prepare_experts_kernel(SortArgs p, const uint16_t* v, int64_t ld,
                                                               int64_t m, int64_t n, uint8_t* q,
                                                               int64_t m_pad, uint8_t* codes, int64_t ldc) {
  if (blockIdx.x == 0) sort_pairs(p);
  else quantise_rows(v, ld, m, n, true, q, m_pad, codes, ldc,
                     (static_cast<int64_t>(blockIdx.x) - 1) * 64 + (threadIdx.x >> 4),
                     (static_cast<int64_t>(gridDim.x) - 1) * 64);
}

// ------------------------------------------------------------------- hosts
struct Plan {
  int32_t bm, bn, splits, per_split;
};

constexpr int64_t kMaxOutputs = 1ll << 36;   // m * n

// Tiles and splits of a product of m x n outputs over kb blocks. Measured, us
// for m x n x k:
//   one split above 128 tiles (1536 x 2048 x 4096, 192 tiles: 43.7, with two
//   44.6; 2048 x 2048 x 4096, 256: 44.4 and 49.1), and with no more than a block
//   for eight tiles from 64 of them on (1024 x 2048 x 2048, 128 tiles: 24.5, with
//   two 28.0; 512 x 2048 x 1024, 64 tiles: 14.2 and 17.7): the steps saved take
//   less than joining;
//   else splits for 256 blocks (1024 x 2048 x 4096, 128 tiles: 33.9 with two, 42.5
//   with one; 512 x 2048 x 4096, 64 tiles: 26.5 with four, 31.4, 40.6; 61 x 3840 x
//   15360, 30 tiles of 64 rows: 23.2 with 8, 31.0 with 4, 22.6 with 15), or 512 of
//   the tiles of 32 rows, of which four fit a CU (20 x 3840 x 15360, 30 tiles: 19.1
//   with 8, 18.5 with 15, 20.9 with 30).
int32_t tile_of_rows(int64_t m) { return m <= 32 ? 32 : m <= 64 ? 64 : 128; }
int64_t splits_of(int64_t m, int64_t n, int64_t kb) {
  const int32_t bm = tile_of_rows(m);
  const int64_t tiles = ((m + bm - 1) / bm) * blocks_of(n);
  int64_t splits = tiles > 128 || (tiles >= 64 && kb <= tiles / 8) ? 1 : (bm == 32 ? 512 : 256) / tiles;
  if (splits > kb / 4) splits = kb / 4;
  return splits < 1 ? 1 : splits;
}
Plan plan_of(int64_t m, int64_t n, int64_t kb) {
  Plan q;
  q.bm = tile_of_rows(m);
  q.bn = 128;
  const int64_t splits = splits_of(m, n, kb);
  int64_t per = (kb + splits - 1) / splits;
  per = (per + 3) / 4 * 4;
  q.per_split = static_cast<int32_t>(per);
  q.splits = static_cast<int32_t>((kb + per - 1) / per);
  if (q.splits < 1) q.splits = 1;
  return q;
}

// Whether a launch stays below 2^32 threads (of at most 512 a block).
bool launchable(const GemmArgs& p) {
  return static_cast<int64_t>(p.mt) * p.nt * (p.order != nullptr ? 8 : p.splits) < (1ll << 23);
}

template <int kScales, bool kExperts>
void launch_gemm(const GemmArgs& p, const Plan& q, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>(static_cast<int64_t>(p.mt) * p.nt * (kExperts ? 8 : p.splits)));
#define BINADE_F8_LAUNCH(BM, BN, WM, WN)                                                              \
  hipLaunchKernelGGL((gemm_kernel<BM, BN, WM, WN, kScales, kExperts>), grid, dim3(64 * WM * WN), 0, st, p)
  if (q.bm == 32) BINADE_F8_LAUNCH(32, 128, 1, 4);
  else if (q.bm == 64) BINADE_F8_LAUNCH(64, 128, 1, 4);
  else BINADE_F8_LAUNCH(128, 128, 2, 2);
#undef BINADE_F8_LAUNCH
}

void launch_kind(int kind, const GemmArgs& p, const Plan& q, hipStream_t st) {
  if (kind == kBlockCode) launch_gemm<kBlockCode, false>(p, q, st);
  else if (kind == kRowCode) launch_gemm<kRowCode, false>(p, q, st);
  else launch_gemm<kBlockF32, false>(p, q, st);
}

// Rows of a quantised operand: tiles of it are read whole. (Of 192 too: the
// workspace's sizes stay what they were.)
int64_t tile_rows(int64_t m) {
  const int64_t a = (m + 127) / 128 * 128, b = (m + 191) / 192 * 192;
  return a > b ? a : b;
}

uint32_t some_blocks(int64_t n) {
  return static_cast<uint32_t>(n < 1 ? 1 : n > 16384 ? 16384 : n);
}

struct Side {   // an operand: its blocks, rows of one, and its codes or scales
  const uint8_t* q;
  const void* scales;
  int64_t rows;
  int32_t ld_scales;
};

int32_t run_product(const Side& x, const Side& w, int kind, int64_t m, int64_t n, int64_t k, void* y,
                    int64_t ldy, bool y_bf16, float* part, hipStream_t st) {
  const int64_t kb = blocks_of(k);
  const Plan q = plan_of(m, n, kb);
  GemmArgs p{};
  p.x = x.q;
  p.x_codes = static_cast<const uint8_t*>(x.scales);
  p.w = w.q;
  p.w_scales = w.scales;
  p.y = y;
  p.part = q.splits > 1 ? part : nullptr;
  p.x_block = x.rows * 128;
  p.w_block = w.rows * 128;
  p.ldy = ldy;
  p.m = m;
  p.n = n;
  p.ld_xc = x.ld_scales;
  p.ld_ws = w.ld_scales;
  p.kb = static_cast<int32_t>(kb);
  p.per_split = q.per_split;
  p.splits = q.splits;
  p.mt = static_cast<int32_t>((m + q.bm - 1) / q.bm);
  p.nt = static_cast<int32_t>((n + q.bn - 1) / q.bn);
  p.y_bf16 = y_bf16;
  const int whole = y_bf16 ? 8 : 4;   // results that a lane stores together
  p.y_vec = n % whole == 0 && ldy % whole == 0 && aligned16(y);
  if (!launchable(p)) return BINADE_EUNSUPPORTED;
  launch_kind(kind, p, q, st);
  if (q.splits > 1) {
    const uint32_t total = static_cast<uint32_t>(m * n), cols = static_cast<uint32_t>(n);
    if (n % 4 == 0)
      hipLaunchKernelGGL(join_kernel<4>, dim3(some_blocks((total / 4 + 255) / 256)), dim3(256), 0, st, part,
                         q.splits, total, cols, y, ldy, y_bf16);
    else
      hipLaunchKernelGGL(join_kernel<1>, dim3(some_blocks((total + 255) / 256)), dim3(256), 0, st, part,
                         q.splits, total, cols, y, ldy, y_bf16);
  }
  return launch_status();
}

// Of the splits' sums: the most that a product of up to m rows takes (fewer rows
// may be split more often), so that a workspace for m serves fewer too.
int64_t part_bytes(int64_t m, int64_t n, int64_t k) {
  const int64_t kb = blocks_of(k);
  int64_t most = 0;
  const auto look = [&](int64_t rows) {
    const Plan q = plan_of(rows, n, kb);
    const int64_t bytes = q.splits > 1 ? up16(4 * q.splits * rows * n) : 0;
    most = bytes > most ? bytes : most;
    return q.splits > 1;
  };
  look(m < 32 ? m : 32);
  if (m > 32) look(m < 64 ? m : 64);
  if (m > 64)   // from one split on, more tiles have one too
    for (int64_t rows = 128; look(rows < m ? rows : m) && rows < m;) rows += 128;
  return most;
}
// The same of a sum over up to m rows (k blocks of 128 of them): the most splits,
// which do not fall as plan_of's own may, a split being whole fours of blocks.
int64_t part_bytes_of_rows(int64_t m, int64_t n, int64_t k) {
  const int64_t kb = blocks_of(m), splits = splits_of(n, k, kb);
  return splits > 1 ? up16(4 * splits * n * k) : 0;
}
int64_t side_bytes(int64_t rows, int64_t cols) {
  return tile_rows(rows) * padded(cols) + up16(tile_rows(rows) * codes_of(cols));
}

int32_t check_f8(const binade_f8* w, bool turned) {
  if (w == nullptr || w->rows < 1 || w->cols < 1 || w->count < 1 || w->values == nullptr ||
      w->scales == nullptr)
    return BINADE_EINVAL;
  if (w->scale_dtype != BINADE_E8M0 && w->scale_dtype != BINADE_F32) return BINADE_EINVAL;
  if (turned && (w->values_t == nullptr || w->scales_t == nullptr)) return BINADE_EINVAL;
  if (w->rows > kMaxSize || w->cols > kMaxSize || w->cols % 32 != 0 || w->count > 65535)
    return BINADE_EUNSUPPORTED;
  if (!aligned16(w->values) || !aligned16(w->scales) || !aligned16(w->values_t) ||
      !aligned16(w->scales_t))
    return BINADE_EUNSUPPORTED;
  return BINADE_OK;
}

bool rows_aligned(const void* p, int64_t ld) { return aligned16(p) && ld % 8 == 0; }

int kind_of(const binade_f8* w) { return w->scale_dtype == BINADE_E8M0 ? kBlockCode : kBlockF32; }

template <int NR, int kWaves>
void launch_few(const SmallArgs& p, int kind, bool experts, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>((p.n + 16 * NR - 1) / (16 * NR)),
                  experts ? static_cast<uint32_t>(p.m) : 1u);
  const dim3 block(64 * kWaves);
  if (experts) {
    if (kind == kBlockCode)
      hipLaunchKernelGGL((few_rows_kernel<NR, kWaves, kBlockCode, true>), grid, block, 0, st, p);
    else
      hipLaunchKernelGGL((few_rows_kernel<NR, kWaves, kBlockF32, true>), grid, block, 0, st, p);
  } else {
    if (kind == kBlockCode)
      hipLaunchKernelGGL((few_rows_kernel<NR, kWaves, kBlockCode, false>), grid, block, 0, st, p);
    else
      hipLaunchKernelGGL((few_rows_kernel<NR, kWaves, kBlockF32, false>), grid, block, 0, st, p);
  }
}

// Whether the experts' products go through the few-row kernel: pairs few
// enough to be looked through by every block.
bool few_pairs(int64_t pairs, int64_t n) { return pairs <= kSmallPairs && pairs * n < (1ll << 27); }

int32_t expert_tile(int64_t pairs, int32_t experts) {
  const int64_t each = pairs / experts;
  return each <= 32 ? 32 : each <= 64 ? 64 : 128;
}

}  // namespace
}  // namespace binade

using namespace binade;

extern "C" int32_t binade_f8_sizes_of(int64_t rows, int64_t cols, int32_t count, int32_t scale_dtype,
                                      binade_f8_sizes* out) {
  if (out == nullptr || rows < 1 || cols < 1 || count < 1 ||
      (scale_dtype != BINADE_E8M0 && scale_dtype != BINADE_F32))
    return BINADE_EINVAL;
  if (rows > kMaxSize || cols > kMaxSize || cols % 32 != 0 || count > 65535) return BINADE_EUNSUPPORTED;
  const uint64_t each = scale_dtype == BINADE_E8M0 ? 1 : 4;
  out->values_bytes = static_cast<uint64_t>(count) * rows * padded(cols);
  out->scales_bytes = static_cast<uint64_t>(count) * blocks_of(rows) * codes_of(cols) * each;
  out->values_t_bytes = static_cast<uint64_t>(count) * cols * padded(rows);
  out->scales_t_bytes = static_cast<uint64_t>(count) * blocks_of(cols) * codes_of(rows) * each;
  return BINADE_OK;
}

extern "C" int32_t binade_f8_pack(const uint16_t* w, binade_f8* out, void* stream) {
  if (out == nullptr || w == nullptr) return BINADE_EINVAL;
  const int32_t rc = check_f8(out, out->values_t != nullptr);
  if (rc != BINADE_OK) return rc;
  if (out->scale_dtype != BINADE_E8M0) return BINADE_EINVAL;
  if (!aligned16(w)) return BINADE_EUNSUPPORTED;
  const int64_t nb = blocks_of(out->rows), kb = blocks_of(out->cols);
  if (nb * kb * out->count >= (1ll << 24) || nb > 65535) return BINADE_EUNSUPPORTED;
  TileArgs p{};
  p.v = w;
  p.ld = out->cols;
  p.m = out->rows;
  p.n = out->cols;
  p.q = const_cast<uint8_t*>(out->values);
  p.codes = static_cast<uint8_t*>(const_cast<void*>(out->scales));
  p.qt = const_cast<uint8_t*>(out->values_t);
  p.codes_t = static_cast<uint8_t*>(const_cast<void*>(out->scales_t));
  p.m_pad = p.m;
  p.n_pad = p.n;
  p.ldc = codes_of(p.n);
  p.ldct = codes_of(p.m);
  p.v_next = p.m * p.n;
  p.q_next = p.m * padded(p.n);
  p.c_next = nb * p.ldc;
  p.qt_next = p.n * padded(p.m);
  p.ct_next = kb * p.ldct;
  p.vec = true;
  hipLaunchKernelGGL((quantise_tile_kernel<false, true>),
                     dim3(static_cast<uint32_t>(kb), static_cast<uint32_t>(nb),
                          static_cast<uint32_t>(out->count)),
                     dim3(256), 0, static_cast<hipStream_t>(stream), p);
  return launch_status();
}

extern "C" int32_t binade_f8_layout(const uint8_t* values, const void* scales, binade_f8* out,
                                    void* stream) {
  if (out == nullptr || values == nullptr || scales == nullptr) return BINADE_EINVAL;
  const int32_t rc = check_f8(out, out->values_t != nullptr);
  if (rc != BINADE_OK) return rc;
  if (!aligned16(values)) return BINADE_EUNSUPPORTED;
  if (out->scale_dtype == BINADE_F32 && (reinterpret_cast<uintptr_t>(scales) & 3u) != 0)
    return BINADE_EUNSUPPORTED;
  const int64_t nb = blocks_of(out->rows), kb = blocks_of(out->cols);
  if (nb * kb * out->count >= (1ll << 24) || nb > 65535) return BINADE_EUNSUPPORTED;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  LayoutArgs p{};
  p.v = values;
  p.q = const_cast<uint8_t*>(out->values);
  p.qt = const_cast<uint8_t*>(out->values_t);
  p.rows = out->rows;
  p.cols = out->cols;
  hipLaunchKernelGGL(layout_kernel,
                     dim3(static_cast<uint32_t>(kb), static_cast<uint32_t>(nb),
                          static_cast<uint32_t>(out->count)),
                     dim3(256), 0, st, p);
  const dim3 grid(some_blocks((nb * kb * out->count + 255) / 256));
  if (out->scale_dtype == BINADE_E8M0)
    hipLaunchKernelGGL(layout_scales_kernel<uint8_t>, grid, dim3(256), 0, st,
                       static_cast<const uint8_t*>(scales),
                       static_cast<uint8_t*>(const_cast<void*>(out->scales)),
                       static_cast<uint8_t*>(const_cast<void*>(out->scales_t)), out->count, nb, kb);
  else
    hipLaunchKernelGGL(layout_scales_kernel<float>, grid, dim3(256), 0, st,
                       static_cast<const float*>(scales),
                       static_cast<float*>(const_cast<void*>(out->scales)),
                       static_cast<float*>(const_cast<void*>(out->scales_t)), out->count, nb, kb);
  return launch_status();
}

extern "C" int64_t binade_f8_gemm_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t) {
  if (m <= kSmallRows || n < 1 || k < 1 || m > kMaxSize || n > kMaxSize || k > kMaxSize) return 0;
  return side_bytes(m, k) + part_bytes(m, n, k);
}

extern "C" int32_t binade_f8_gemm(const binade_f8* w, const uint16_t* x, int64_t m, int64_t ldx,
                                  void* y, int64_t ldy, int32_t y_dtype, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
  const int32_t rc = check_f8(w, false);
  if (rc != BINADE_OK) return rc;
  if (w->count != 1 || m < 0 || (y_dtype != BINADE_F32 && y_dtype != BINADE_BF16)) return BINADE_EINVAL;
  if (m == 0) return BINADE_OK;
  const int64_t n = w->rows, k = w->cols;
  if (x == nullptr || y == nullptr || ldx < k || ldy < n) return BINADE_EINVAL;
  if (!rows_aligned(x, ldx) || m > kMaxSize || ldx > (1 << 24) || ldy > (1 << 24) || m * n > kMaxOutputs)
    return BINADE_EUNSUPPORTED;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (m <= kSmallRows) {
    SmallArgs p{};
    p.x = x;
    p.w = w->values;
    p.w_scales = w->scales;
    p.y = y;
    p.ldx = ldx;
    p.ldy = ldy;
    p.n = n;
    p.k = k;
    p.m = static_cast<int32_t>(m);
    p.ld_ws = static_cast<int32_t>(codes_of(k));
    p.y_bf16 = y_dtype == BINADE_BF16;
    launch_few<1, 8>(p, kind_of(w), false, st);
    return launch_status();
  }
  if (workspace == nullptr || workspace_bytes < binade_f8_gemm_workspace_bytes(m, n, k, y_dtype))
    return BINADE_ENOSPACE;
  if (!aligned16(workspace)) return BINADE_EUNSUPPORTED;
  uint8_t* q = static_cast<uint8_t*>(workspace);
  uint8_t* codes = q + tile_rows(m) * padded(k);
  float* part = reinterpret_cast<float*>(q + side_bytes(m, k));
  hipLaunchKernelGGL(quantise_rows_kernel, dim3(some_blocks((m * blocks_of(k) + 15) / 16)), dim3(256),
                     0, st, x, ldx, m, k, true, q, tile_rows(m), codes, codes_of(k));
  return run_product({q, codes, tile_rows(m), static_cast<int32_t>(codes_of(k))},
                     {w->values, w->scales, n, static_cast<int32_t>(codes_of(k))}, kind_of(w),
                     m, n, k, y, ldy, y_dtype == BINADE_BF16, part, st);
}

extern "C" int64_t binade_f8_gemm_grad_workspace_bytes(int64_t m, int64_t n, int64_t k,
                                                       int32_t need_dx, int32_t need_dw, int32_t) {
  if (m < 1 || n < 1 || k < 1 || m > kMaxSize || n > kMaxSize || k > kMaxSize) return 0;
  int64_t bytes = 0, part = 0;
  if (need_dx) {
    bytes += side_bytes(m, n);
    part = part_bytes(m, k, n);
  }
  if (need_dw) {
    bytes += side_bytes(n, m) + side_bytes(k, m);
    const int64_t b = part_bytes_of_rows(m, n, k);
    part = b > part ? b : part;
  }
  return bytes + part;
}

extern "C" int32_t binade_f8_gemm_grad(const binade_f8* w, const uint16_t* x, int64_t m, int64_t ldx,
                                       const uint16_t* dy, int64_t ld_dy, uint16_t* dx, int64_t ld_dx,
                                       void* dw, int32_t dw_dtype, void* workspace,
                                       int64_t workspace_bytes, void* stream) {
  const bool need_dx = dx != nullptr, need_dw = dw != nullptr;
  const int32_t rc = check_f8(w, need_dx);
  if (rc != BINADE_OK) return rc;
  if (w->count != 1 || m < 0 || (dw_dtype != BINADE_F32 && dw_dtype != BINADE_BF16)) return BINADE_EINVAL;
  const int64_t n = w->rows, k = w->cols;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (m > 0 && (dy == nullptr || ld_dy < n || (need_dx && ld_dx < k) ||
                (need_dw && (x == nullptr || ldx < k))))
    return BINADE_EINVAL;
  if (m > kMaxSize || ld_dy > (1 << 24) || (need_dx && ld_dx > (1 << 24)) ||
      (need_dw && ldx > (1 << 24)) || m * k > kMaxOutputs || n * k > kMaxOutputs ||
      m * n > kMaxOutputs)
    return BINADE_EUNSUPPORTED;
  if (need_dw && m > 0 && !rows_aligned(x, ldx)) return BINADE_EUNSUPPORTED;
  if (m == 0) {
    if (need_dw) {
      const int64_t words = n * k / (dw_dtype == BINADE_F32 ? 1 : 2);   // k is even
      hipLaunchKernelGGL(zero_kernel, dim3(some_blocks((words + 255) / 256)), dim3(256), 0, st,
                         static_cast<uint32_t*>(dw), words);
    }
    return launch_status();
  }
  if (!need_dx && !need_dw) return BINADE_OK;
  if (workspace == nullptr ||
      workspace_bytes < binade_f8_gemm_grad_workspace_bytes(m, n, k, need_dx, need_dw, dw_dtype))
    return BINADE_ENOSPACE;
  if (!aligned16(workspace)) return BINADE_EUNSUPPORTED;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  const auto take = [&](int64_t rows, int64_t cols) {
    Side s{at, at + tile_rows(rows) * padded(cols), tile_rows(rows), static_cast<int32_t>(codes_of(cols))};
    at += side_bytes(rows, cols);
    return s;
  };
  Side dy_rows{}, dy_cols{}, x_cols{};
  if (need_dx) dy_rows = take(m, n);
  if (need_dw) {
    dy_cols = take(n, m);
    x_cols = take(k, m);
  }
  float* part = reinterpret_cast<float*>(at);
  const bool vec = n % 8 == 0 && rows_aligned(dy, ld_dy);
  const auto turn = [&](const uint16_t* v, int64_t ld, int64_t cols, bool v8, const Side* rows_side,
                        const Side& cols_side) {
    TileArgs p{};
    p.v = v;
    p.ld = ld;
    p.m = m;
    p.n = cols;
    p.qt = const_cast<uint8_t*>(cols_side.q);
    p.codes_t = static_cast<uint8_t*>(const_cast<void*>(cols_side.scales));
    p.n_pad = cols_side.rows;
    p.ldct = cols_side.ld_scales;
    p.vec = v8;
    const dim3 grid(static_cast<uint32_t>(blocks_of(cols)), static_cast<uint32_t>(blocks_of(m)), 1);
    if (rows_side != nullptr) {
      p.q = const_cast<uint8_t*>(rows_side->q);
      p.codes = static_cast<uint8_t*>(const_cast<void*>(rows_side->scales));
      p.m_pad = rows_side->rows;
      p.ldc = rows_side->ld_scales;
      hipLaunchKernelGGL((quantise_tile_kernel<true, false>), grid, dim3(256), 0, st, p);
    } else {
      hipLaunchKernelGGL((quantise_tile_kernel<false, false>), grid, dim3(256), 0, st, p);
    }
  };
  if (need_dw) {
    turn(dy, ld_dy, n, vec, need_dx ? &dy_rows : nullptr, dy_cols);
    turn(x, ldx, k, true, nullptr, x_cols);
  } else {
    hipLaunchKernelGGL(quantise_rows_kernel, dim3(some_blocks((m * blocks_of(n) + 15) / 16)), dim3(256),
                       0, st, dy, ld_dy, m, n, vec, const_cast<uint8_t*>(dy_rows.q), dy_rows.rows,
                       static_cast<uint8_t*>(const_cast<void*>(dy_rows.scales)),
                       static_cast<int64_t>(dy_rows.ld_scales));
  }
  int32_t status = launch_status();
  if (status != BINADE_OK) return status;
  if (need_dx) {
    status = run_product(dy_rows, {w->values_t, w->scales_t, k, static_cast<int32_t>(codes_of(n))},
                         kind_of(w), m, k, n, dx, ld_dx, true, part, st);
    if (status != BINADE_OK) return status;
  }
  if (need_dw)
    status = run_product(dy_cols, x_cols, kRowCode, n, k, m, dw, k, dw_dtype == BINADE_BF16, part, st);
  return status;
}

namespace {
struct ExpertSpace {
  int64_t order, tiles, total;   // bytes before each, and of all
  int64_t share;                 // places of tiles of an XCD
};
ExpertSpace expert_space(int64_t rows, int64_t pairs, int64_t k, int32_t experts) {
  ExpertSpace s;
  const int32_t bm = expert_tile(pairs, experts);
  const int64_t each = experts + 1 < pairs ? experts + 1 : pairs;   // experts with a part of a tile
  s.share = (pairs / bm + each) / 8 + 2;   // two parts, each rounded up
  s.order = side_bytes(rows, k);
  s.tiles = s.order + up16(4 * pairs);
  // with smaller tiles, as fewer pairs have them, there are more: a workspace
  // for these pairs serves fewer too
  int64_t most = s.share;
  for (const int32_t small : {32, 64}) {
    if (small >= bm) break;
    const int64_t p = (small + 1ll) * experts - 1, e = experts + 1 < p ? experts + 1 : p;   // the most pairs of them
    most = (p / small + e) / 8 + 2 > most ? (p / small + e) / 8 + 2 : most;
  }
  s.total = s.tiles + 16 * 8 * most;
  return s;
}
}  // namespace

extern "C" int64_t binade_f8_moe_workspace_bytes(int64_t n_tokens, int32_t top_k, int32_t x_per_slot,
                                                 int32_t n_experts, int64_t n, int64_t k) {
  if (n_tokens < 1 || top_k < 1 || top_k > 64 || n_tokens > kMaxPairs || n_experts < 1 ||
      n_experts > kMaxExperts || n < 1 || k < 1 || n_tokens * top_k > kMaxPairs || n > kMaxSize ||
      k > kMaxSize)
    return 0;
  const int64_t pairs = n_tokens * top_k;
  if (few_pairs(pairs, n)) return 0;
  return expert_space(x_per_slot ? pairs : n_tokens, pairs, k, n_experts).total;
}

extern "C" int32_t binade_f8_moe_gemm(const binade_f8* experts, const uint16_t* x, int64_t ldx,
                                      int32_t x_per_slot, const int32_t* idx, int64_t n_tokens,
                                      int32_t top_k, void* y, int64_t ldy, int32_t y_dtype,
                                      void* workspace, int64_t workspace_bytes, uint32_t* dev_status,
                                      void* stream) {
  const int32_t rc = check_f8(experts, false);
  if (rc != BINADE_OK) return rc;
  if (n_tokens < 0 || top_k < 1 || top_k > 64 || (y_dtype != BINADE_F32 && y_dtype != BINADE_BF16))
    return BINADE_EINVAL;
  if (n_tokens == 0) return BINADE_OK;
  const int64_t n = experts->rows, k = experts->cols;
  if (x == nullptr || idx == nullptr || y == nullptr || ldx < k || ldy < n) return BINADE_EINVAL;
  if (!rows_aligned(x, ldx) || ldx > (1 << 24) || ldy > (1 << 24) || experts->count > kMaxExperts ||
      n_tokens > kMaxPairs || n_tokens * top_k > kMaxPairs || n_tokens * top_k * n > kMaxOutputs)
    return BINADE_EUNSUPPORTED;
  const int64_t pairs = n_tokens * top_k;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t w_next = n * padded(k), s_next = blocks_of(n) * codes_of(k);
  const int32_t per_row = x_per_slot ? 1 : top_k;
  if (few_pairs(pairs, n)) {
    SmallArgs p{};
    p.x = x;
    p.w = experts->values;
    p.w_scales = experts->scales;
    p.y = y;
    p.ldx = ldx;
    p.ldy = ldy;
    p.n = n;
    p.k = k;
    p.m = static_cast<int32_t>(pairs);
    p.ld_ws = static_cast<int32_t>(codes_of(k));
    p.y_bf16 = y_dtype == BINADE_BF16;
    p.idx = idx;
    p.status = dev_status;
    p.w_next = w_next;
    p.s_next = s_next;
    p.n_experts = experts->count;
    p.pairs_a_row = per_row;
    launch_few<2, 8>(p, kind_of(experts), true, st);
    return launch_status();
  }
  const int64_t rows = x_per_slot ? pairs : n_tokens;
  if (workspace == nullptr ||
      workspace_bytes < binade_f8_moe_workspace_bytes(n_tokens, top_k, x_per_slot, experts->count, n, k))
    return BINADE_ENOSPACE;
  if (!aligned16(workspace)) return BINADE_EUNSUPPORTED;
  const ExpertSpace space = expert_space(rows, pairs, k, experts->count);
  uint8_t* at = static_cast<uint8_t*>(workspace);
  uint8_t* codes = at + tile_rows(rows) * padded(k);
  Plan q{};
  q.bm = expert_tile(pairs, experts->count);
  q.bn = 128;
  q.splits = 1;
  GemmArgs p{};
  p.order = reinterpret_cast<int32_t*>(at + space.order);
  p.tiles = reinterpret_cast<int4*>(at + space.tiles);
  p.mt = static_cast<int32_t>(space.share);
  p.nt = static_cast<int32_t>((n + 127) / 128);
  p.splits = 1;
  if (!launchable(p)) return BINADE_EUNSUPPORTED;
  const SortArgs sort{idx, static_cast<int32_t>(pairs), experts->count, q.bm, p.mt,
                      const_cast<int32_t*>(p.order), const_cast<int4*>(p.tiles), dev_status};
  const int64_t blocks = (rows * blocks_of(k) + 127) / 128;   // two blocks of a row a thread
  hipLaunchKernelGGL(prepare_experts_kernel, dim3(1 + some_blocks(blocks)), dim3(1024), 0, st, sort, x, ldx,
                     rows, k, at, tile_rows(rows), codes, codes_of(k));
  p.x = at;
  p.x_codes = codes;
  p.w = experts->values;
  p.w_scales = experts->scales;
  p.y = y;
  p.x_block = tile_rows(rows) * 128;
  p.w_block = n * 128;
  p.ldy = ldy;
  p.m = pairs;
  p.n = n;
  p.ld_xc = static_cast<int32_t>(codes_of(k));
  p.ld_ws = static_cast<int32_t>(codes_of(k));
  p.kb = static_cast<int32_t>(blocks_of(k));
  p.per_split = (p.kb + 3) / 4 * 4;
  p.y_bf16 = y_dtype == BINADE_BF16;
  const int whole = p.y_bf16 ? 8 : 4;
  p.y_vec = n % whole == 0 && ldy % whole == 0 && aligned16(y);
  p.w_next = w_next;
  p.s_next = s_next;
  p.pairs_a_row = per_row;
  if (kind_of(experts) == kBlockCode) launch_gemm<kBlockCode, true>(p, q, st);
  else launch_gemm<kBlockF32, true>(p, q, st);
  return launch_status();
}
