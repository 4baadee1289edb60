// What the two routers (moe_route.hip: by logits, moe_route_scored.hip: by
// scores) share: steps across a row's lanes, logits, ordered keys and their
// sorting, and the sums over rows.
#ifndef BINADE_MOE_ROUTE_H
#define BINADE_MOE_ROUTE_H

#include <hip/hip_runtime.h>

#include <type_traits>

#include "binade.h"
#include "device_common.h"

namespace binade {
namespace {

using namespace dev;

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
constexpr int kSorted = 8;        // slots the sorting choice fills
constexpr int64_t kHead = 192;    // bytes of a workspace before these: ticket, shares of the loss

// ------------------------------------------------------ steps across lanes
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), kCtrl, 0xF, 0xF,
                                                           true));
}

// The value of the lane's partner in step kStep of a butterfly over lanes
// (1, 2, 4, 8, 16, 32 apart; mirrors stand for 4 and 8: all lanes of a half
// hold the same by then). Both lanes of a pair get the pair as (a, b) in one
// order, so that what they make of it is the same bits.
template <int kStep>
__device__ __forceinline__ void pair_of(uint32_t v, uint32_t& a, uint32_t& b) {
  if (kStep == 16 || kStep == 32) {
    const auto r = kStep == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                               : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = r[0];
    b = r[1];
    return;
  }
  a = v;
  b = kStep == 1 ? dpp<0xB1>(v)      // quad_perm 1 0 3 2
      : kStep == 2 ? dpp<0x4E>(v)    // quad_perm 2 3 0 1
      : kStep == 4 ? dpp<0x141>(v)   // row_half_mirror
                   : dpp<0x140>(v);  // row_mirror
}

template <int kStep>
__device__ __forceinline__ void pair_of(uint64_t v, uint64_t& a, uint64_t& b) {
  uint32_t a0, a1, b0, b1;
  pair_of<kStep>(static_cast<uint32_t>(v), a0, b0);
  pair_of<kStep>(static_cast<uint32_t>(v >> 32), a1, b1);
  a = (static_cast<uint64_t>(a1) << 32) | a0;
  b = (static_cast<uint64_t>(b1) << 32) | b0;
}

template <int kStep>
__device__ __forceinline__ void pair_of(int32_t v, int32_t& a, int32_t& b) {
  uint32_t c, d;
  pair_of<kStep>(static_cast<uint32_t>(v), c, d);
  a = static_cast<int32_t>(c);
  b = static_cast<int32_t>(d);
}

template <int G, int kStep = 1, typename F>
__device__ __forceinline__ void butterfly(F f) {
  if constexpr (kStep < G) {
    f(std::integral_constant<int, kStep>());
    butterfly<G, 2 * kStep>(f);
  }
}

// a + b = b + a: every lane of a group ends with the same bits.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  butterfly<G>([&](auto step) {
    uint32_t a, b;
    pair_of<decltype(step)::value>(__float_as_uint(v), a, b);
    v = __uint_as_float(a) + __uint_as_float(b);
  });
  return v;
}

template <int G>
__device__ __forceinline__ float group_max(float v) {
  butterfly<G>([&](auto step) {
    uint32_t a, b;
    pair_of<decltype(step)::value>(__float_as_uint(v), a, b);
    v = fmaxf(__uint_as_float(a), __uint_as_float(b));
  });
  return v;
}

template <int G, typename Key>
__device__ __forceinline__ Key group_max_key(Key v) {
  butterfly<G>([&](auto step) {
    Key a, b;
    pair_of<decltype(step)::value>(v, a, b);
    v = a > b ? a : b;
  });
  return v;
}

// ------------------------------------------------------------------ logits
// V logits of a row from expert e0 on, as they are; -inf behind the last
// expert. vec: rows and their length are whole 16-byte pieces.
template <int V, bool kBf16>
struct Logits {
  uint32_t d[kBf16 ? V / 2 : V];

  __device__ __forceinline__ void load(const void* p, int64_t row, int32_t e0, int32_t n, bool vec) {
    constexpr int kPiece = kBf16 ? 4 : 8;   // dwords of 8 logits
    constexpr uint32_t kNone = kBf16 ? 0xFF80FF80u : 0xFF800000u;
    if (vec) {
#pragma unroll
      for (int b = 0; b < V / 8; ++b) {
        const int64_t at = row + (e0 + 8 * b < n ? e0 + 8 * b : 0);
        const void* from = kBf16 ? static_cast<const void*>(static_cast<const uint16_t*>(p) + at)
                                 : static_cast<const void*>(static_cast<const float*>(p) + at);
        __builtin_memcpy(&d[kPiece * b], __builtin_assume_aligned(from, 16), 4 * kPiece);
      }
#pragma unroll
      for (int b = 0; b < V / 8; ++b)
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
          d[kPiece * b + j] = e0 + 8 * b < n ? d[kPiece * b + j] : kNone;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int64_t at = row + (e0 + j < n ? e0 + j : 0);
        if (kBf16) {
          const uint32_t u = e0 + j < n ? static_cast<const uint16_t*>(p)[at] : kNone & 0xFFFFu;
          d[j / 2] = j & 1 ? d[j / 2] | (u << 16) : u;
        } else {
          d[j] = e0 + j < n ? static_cast<const uint32_t*>(p)[at] : kNone;
        }
      }
    }
  }

  __device__ __forceinline__ float value(int j) const {
    return kBf16 ? (j & 1 ? bf16_hi(d[j / 2]) : bf16_lo(d[j / 2])) : __uint_as_float(d[j]);
  }
};

// -------------------------------------------------------------------- keys
// Ordered form of a logit's bits: rising with the value, -0 as +0 (for a
// negative one the two's complement of its bits); -inf and NaN of either sign
// lie outside (kLow, kHigh].
struct KeyBf16 {
  typedef uint32_t Key;
  static constexpr uint32_t kLow = 0x0080u, kHigh = 0xFF80u;   // of -inf, of +inf
  template <int V, bool kClean>
  static __device__ __forceinline__ void make(const Logits<V, true>& x, int32_t e0, Key (&key)[V]) {
    typedef short short2v __attribute__((ext_vector_type(2)));
    typedef unsigned short ushort2v __attribute__((ext_vector_type(2)));
    const uint32_t last = 0xFFFFu - static_cast<uint32_t>(e0);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {   // two at a time
      const uint32_t neg = __builtin_bit_cast(uint32_t, __builtin_bit_cast(short2v, x.d[j]) >> 15);
      const uint32_t add = (neg & 0x00010001u) | (~neg & 0x80008000u);
      const uint32_t o = __builtin_bit_cast(
          uint32_t, __builtin_bit_cast(ushort2v, x.d[j] ^ neg) + __builtin_bit_cast(ushort2v, add));
      uint32_t lo = o << 16, hi = o & 0xFFFF0000u;
      if (kClean) {
        lo = lo > (kHigh << 16) ? 0u : lo;
        hi = hi > (kHigh << 16) ? 0u : hi;
      }
      key[2 * j] = lo | (last - 2 * j);
      key[2 * j + 1] = hi | (last - 2 * j - 1);
    }
  }
  static __device__ __forceinline__ uint32_t order_of(Key k) { return k >> 16; }
  static __device__ __forceinline__ int32_t expert(Key k) {
    return static_cast<int32_t>(0xFFFFu - (k & 0xFFFFu));
  }
  static __device__ __forceinline__ float value(Key k) {
    const uint32_t o = k >> 16;
    return __uint_as_float((o & 0x8000u ? o - 0x8000u : 0x10000u - o) << 16);
  }
};

struct KeyF32 {
  typedef uint64_t Key;
  static constexpr uint32_t kLow = 0x00800000u, kHigh = 0xFF800000u;
  template <int V, bool kClean>
  static __device__ __forceinline__ void make(const Logits<V, false>& x, int32_t e0,
                                              Key (&key)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t neg = static_cast<uint32_t>(static_cast<int32_t>(x.d[j]) >> 31);
      uint32_t o = (x.d[j] ^ neg) + ((neg & 1u) | (~neg & 0x80000000u));
      if (kClean) o = o > kHigh ? 0u : o;
      key[j] = (static_cast<uint64_t>(o) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(e0 + j));
    }
  }
  static __device__ __forceinline__ uint32_t order_of(Key k) {
    return static_cast<uint32_t>(k >> 32);
  }
  static __device__ __forceinline__ int32_t expert(Key k) {
    return static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(k));
  }
  static __device__ __forceinline__ float value(Key k) {
    const uint32_t o = order_of(k);
    return __uint_as_float(o & 0x80000000u ? o - 0x80000000u : 0u - o);
  }
};

template <typename Key>
__device__ __forceinline__ void exchange(Key& a, Key& b) {   // the larger first
  const Key hi = a > b ? a : b, lo = a > b ? b : a;
  a = hi;
  b = lo;
}

template <typename Key>
__device__ __forceinline__ void sort8(Key* k) {   // 19 exchanges, falling
  constexpr int net[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6},
                              {5, 7}, {1, 2}, {5, 6}, {0, 4}, {3, 7}, {1, 5}, {2, 6},
                              {1, 4}, {3, 6}, {2, 4}, {3, 5}, {3, 4}};
#pragma unroll
  for (int j = 0; j < 19; ++j) exchange(k[net[j][0]], k[net[j][1]]);
}

template <typename Key>
__device__ __forceinline__ void sort_bitonic8(Key* k) {
#pragma unroll
  for (int d = 4; d >= 1; d >>= 1)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if ((j & d) == 0) exchange(k[j], k[j + d]);
}

// The group's best eight keys, falling, in every lane.
template <int G, int V, typename Key>
__device__ __forceinline__ void best8(const Key (&key)[V], Key (&best)[8]) {
#pragma unroll
  for (int b = 0; b < V / 8; ++b) {
    Key k[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) k[j] = key[8 * b + j];
    sort8(k);
    if (b == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) best[j] = k[j];
    } else {
      Key m[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = best[j] > k[7 - j] ? best[j] : k[7 - j];
      sort_bitonic8(m);
#pragma unroll
      for (int j = 0; j < 8; ++j) best[j] = m[j];
    }
  }
  butterfly<G>([&](auto step) {
    Key a[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) pair_of<decltype(step)::value>(best[j], a[j], b[j]);
#pragma unroll
    for (int j = 0; j < 8; ++j) best[j] = a[j] > b[7 - j] ? a[j] : b[7 - j];
    sort_bitonic8(best);
  });
}

// ------------------------------------------------------------------ values
// exp(d) for d <= 0 (-inf: 0), or NaN. log2 e is taken as the sum of two fp32:
// the first alone is 1.3e-8 too small, which moves every small probability the
// same way. What is left is the product's rounding, |d| 2^-24 of the value to
// either side, as much as that of the difference d itself.
__device__ __forceinline__ float exp_of(float d) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(d, 1.44269502e+0f, d * 1.92596303e-8f));
}

// 1 / v within 2^-24 and a little: a Newton step behind the instruction, which
// is one step off. v is at least 2^-10 here; 0 (a row that does not count)
// gives NaN, which nothing takes.
__device__ __forceinline__ float inverse(float v) {
  const float r = __builtin_amdgcn_rcpf(v);
  return __builtin_fmaf(__builtin_fmaf(-v, r, 1.0f), r, r);
}

// ----------------------------------------------------------- sums over rows
struct RouteArgs {
  const void* logits;
  const uint8_t* valid;
  int32_t* idx;
  float* weights;
  int32_t* counts;        // [n_experts + 1], or NULL: no sums over rows
  float* prob_sum;
  float* loss;
  int32_t* part_counts;   // [blocks, n_experts + 1]
  float* part_prob;       // [blocks, n_experts]
  double* part_loss;      // [16] of route_stats_kernel's blocks
  uint32_t* ticket;       // of the same: which block is the last
  int64_t ld, n_tokens;
  int32_t n_experts, top_k;
  bool renorm, vec;
};

// Sums over waves, blocks and experts run in fp64: there are few, and a chain
// of 16 or 32 fp32 additions of like size would cost the summed probabilities
// and the loss more than everything before it (2048 tokens of 128 experts:
// 6.1e-8 off in place of 2.7e-8).

// The sum of a block's values by a fixed tree, in thread 0. Whole waves.
__device__ __forceinline__ double block_sum(double v, double* red) {
  butterfly<64>([&](auto step) {
    uint64_t a, b;
    pair_of<decltype(step)::value>(__builtin_bit_cast(uint64_t, v), a, b);
    v = __builtin_bit_cast(double, a) + __builtin_bit_cast(double, b);
  });
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double sum = 0.0;
  if (threadIdx.x == 0)
    for (uint32_t w = 0; w < blockDim.x / 64; ++w) sum += red[w];
  return sum;
}

// The loss from sum_e counts[e] * prob_sum[e].
__device__ __forceinline__ float loss_of(double sum, int32_t n_experts, int32_t top_k,
                                         int32_t rows) {
  const double r = rows > 0 ? rows : 1;
  return static_cast<float>(n_experts * sum / (top_k * r * r));
}

// Adds the blocks' partial counts and sums: a block has 64 experts side by
// side and 16 rows of partial sums at a time, in a fixed order. The last block
// to end adds the blocks' shares of the loss, in block order.
__global__ __launch_bounds__(1024) void route_stats_kernel(RouteArgs p, int32_t blocks) {
  __shared__ int32_t count_s[16][64];
  __shared__ double sum_s[16][64];
  __shared__ double red[16];
  __shared__ int32_t rows_s;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t e = blockIdx.x * 64 + lane;
  if (wave == 0) {
    int32_t rows = 0;
    for (int32_t b = lane; b < blocks; b += 64)
      rows += p.part_counts[static_cast<int64_t>(b) * (p.n_experts + 1) + p.n_experts];
    for (int s = 32; s >= 1; s >>= 1) rows += __shfl_xor(rows, s, 64);
    if (lane == 0) rows_s = rows;
  }
  int32_t c = 0;
  double s = 0.0;
  if (e < p.n_experts) {
    constexpr int kAhead = 16;   // rows of partial sums on their way at once
    const int32_t* pc = p.part_counts + e;
    const float* pp = p.part_prob + e;
    int32_t b = wave;
    for (; b + (kAhead - 1) * 16 < blocks; b += kAhead * 16) {
      int32_t cs[kAhead];
      float ss[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        cs[j] = pc[static_cast<int64_t>(b + j * 16) * (p.n_experts + 1)];
        ss[j] = pp[static_cast<int64_t>(b + j * 16) * p.n_experts];
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        c += cs[j];
        s += ss[j];
      }
    }
#pragma unroll 4
    for (; b < blocks; b += 16) {
      c += pc[static_cast<int64_t>(b) * (p.n_experts + 1)];
      s += pp[static_cast<int64_t>(b) * p.n_experts];
    }
  }
  count_s[wave][lane] = c;
  sum_s[wave][lane] = s;
  __syncthreads();
  double term = 0.0;
  if (wave == 0 && e < p.n_experts) {
    for (int q = 1; q < 16; ++q) {
      c += count_s[q][lane];
      s += sum_s[q][lane];
    }
    p.counts[e] = c;
    p.prob_sum[e] = static_cast<float>(s);
    term = c * s;
  }
  term = block_sum(term, red);
  if (threadIdx.x != 0) return;
  if (blockIdx.x == 0) p.counts[p.n_experts] = rows_s;
  if (gridDim.x > 1) {
    p.part_loss[blockIdx.x] = term;
    __threadfence();
    if (atomicAdd(p.ticket, 1u) != gridDim.x - 1) return;
    __threadfence();
    term = 0.0;
    for (uint32_t b = 0; b < gridDim.x; ++b)
      term += __hip_atomic_load(p.part_loss + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  p.loss[0] = loss_of(term, p.n_experts, p.top_k, rows_s);
}

// ------------------------------------------------------------------- hosts
bool route_sizes_ok(int64_t n_tokens, int32_t n_experts) {
  return n_tokens >= 0 && n_tokens <= (1ll << 30) && n_experts >= 1 && n_experts <= kMaxExperts;
}

// Whether rows of n at stride ld from p are whole 16-byte pieces of 8 values.
bool whole_pieces(const void* p, int32_t n, int64_t ld, bool bf16) {
  return aligned16(p) && n % 8 == 0 && ld % (bf16 ? 8 : 4) == 0;
}

}  // namespace
}  // namespace binade

#endif
