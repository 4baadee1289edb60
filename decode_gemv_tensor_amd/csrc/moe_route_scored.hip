// The router by scores and its backward: sigmoid or softmax scores, a bias for
// balance, groups of experts, top-k of the best groups, scaled weights (the
// arithmetic is stated in binade.h). Rows, lanes and sums over rows as in
// moe_route.hip: a row belongs to G lanes with V adjacent experts each.
//
// Choice. What is compared is score + bias in fp64. Nearly every row is
// settled in fp32: its values become 32-bit keys that max and min alone sort,
// and the row counts as settled if every gap that decides something (between
// the slots, to the best expert left out, between the last group taken and the
// first left out) is larger than the fp32 values can be off. A wave with a row
// that is not settled works its rows out again in fp64. Without bias the
// logits themselves are the order, which is exact: bf16 ones with the expert
// in the key's other half, so that ties are settled too. The slots' experts
// are found by their values: a lane looks for its own among the sorted ones.
//
// Bound by vector instructions: 1376 for four rows of 256 experts (16 scores, a
// sort of 16 and four merges of eight a lane, groups, the checks of gaps);
// 65536 rows 65 us, of which 71 MB are 14. Three waves a SIMD instead of two
// (168 registers, with spills) take as long.
//
// Scores relative to the row's largest: sigmoid(x) = exp(min(x, 0)) / (1 +
// exp(-|x|)), and quotients of scores do not change when exp(min(x, 0)) is
// taken as exp(min(x, 0) - c) with c = min(0, the largest x); so neither sums
// of scores nor their quotients underflow, however low a row's logits are.
#include "moe_route.h"

namespace binade {
namespace {

constexpr int kWavesABlock = 4;
constexpr int32_t kScoredBlocks = 512;   // at most: each leaves one row of partial sums
constexpr int kMaxGroups = 64;

struct ScoredArgs {
  RouteArgs r;
  const float* bias;
  int32_t groups, group_size, top_groups, group_best;
  int32_t lanes_a_group;   // a power of two of whole lanes, or 0
  int32_t parts;           // otherwise: lanes that look through a group in LDS
  float scale;
  bool sigmoid;
};

// exp(-|x|).
__device__ __forceinline__ float low_exp(float x) { return exp_of(-fabsf(x)); }

// KeyF32's order of any value: rising with it, -0 as +0; NaN and -inf as 0
// (never taken).
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v);
  const uint32_t neg = static_cast<uint32_t>(static_cast<int32_t>(b) >> 31);
  const uint32_t o = (b ^ neg) + ((neg & 1u) | (~neg & 0x80000000u));
  return v > -__builtin_inff() ? o : 0u;
}
// A value's bits as a whole number of the same order, and back. -0 would lie
// below +0: values come here as +0 (score + bias is never -0, a logit gets + 0).
// -inf is the least.
constexpr int32_t kNone = static_cast<int32_t>(0x807FFFFFu);   // of -inf
__device__ __forceinline__ int32_t ordered(float v) {
  const int32_t b = __float_as_int(v);
  return b ^ static_cast<int32_t>(static_cast<uint32_t>(b >> 31) >> 1);
}
__device__ __forceinline__ float value_of(int32_t o) {
  return __int_as_float(o ^ static_cast<int32_t>(static_cast<uint32_t>(o >> 31) >> 1));
}

// How far apart two fp32 values of at most |v| have to be for their order to
// be the exact one: `base` for their scores and 2 u |v| for the two additions of
// a bias. u = 2^-24. A sigmoid errs by at most 4 u (an exponential, of at most
// (2 |x| + 2) u relative, the sum, its inverse and the product): base is 16 u. A
// softmax p = exp(d) / total errs by (2 |d| + 2) u p and by its total, which all
// of the row have in common: 21 u relative from up to 15 additions a lane and
// 6 across lanes, 11 u from its terms ((2 |d| + 2) u on the average that 1024 of
// them can bring), 1 u from the inverse. That is below 40 u of the row's largest
// p: base is 80 u of it, and of 1 / total, which is no less.
constexpr float kSigmoidBase = 9.5367432e-7f, kSoftmaxBase = 4.7683716e-6f;
__device__ __forceinline__ float apart(float base, float v) { return base + 1.1920929e-7f * fabsf(v); }

// The two largest of a lane's and its partner's two.
template <int kStep, typename T>
__device__ __forceinline__ void join_two(T& a, T& b) {
  T a0, a1, b0, b1;
  if constexpr (sizeof(T) == 4) {
    uint32_t x, y;
    pair_of<kStep>(__builtin_bit_cast(uint32_t, a), x, y);
    a0 = __builtin_bit_cast(T, x), a1 = __builtin_bit_cast(T, y);
    pair_of<kStep>(__builtin_bit_cast(uint32_t, b), x, y);
    b0 = __builtin_bit_cast(T, x), b1 = __builtin_bit_cast(T, y);
  } else {
    uint64_t x, y;
    pair_of<kStep>(__builtin_bit_cast(uint64_t, a), x, y);
    a0 = __builtin_bit_cast(T, x), a1 = __builtin_bit_cast(T, y);
    pair_of<kStep>(__builtin_bit_cast(uint64_t, b), x, y);
    b0 = __builtin_bit_cast(T, x), b1 = __builtin_bit_cast(T, y);
  }
  const T low = a0 > a1 ? a1 : a0, second = b0 > b1 ? b0 : b1;
  a = a0 > a1 ? a0 : a1;
  b = low > second ? low : second;
}

// A group's score in fp32, and how far it may be off: by its two terms' errors,
// which go by their magnitudes, and the sum's rounding, below both together.
// Terms of opposite sign cancel in the score and not in this.
struct GroupScore {
  float v, off;
};
__device__ __forceinline__ float number(GroupScore s) { return s.v; }
__device__ __forceinline__ double number(double s) { return s; }

// The score of a group whose two largest are a >= b (-inf: none). An infinite
// one is exact; where the sum alone overflows, `off` is infinite.
__device__ __forceinline__ GroupScore score_of(const ScoredArgs& p, float a, float b, bool exact, float base) {
  const bool two = p.group_best == 2 && b > -__builtin_inff();
  return {two ? a + b : a,
          exact || !(fabsf(a) < __builtin_inff()) ? 0.0f : apart(base, fabsf(a) + (two ? fabsf(b) : 0.0f))};
}
__device__ __forceinline__ double score_of(const ScoredArgs& p, double a, double b, bool, float) {
  return p.group_best == 2 && b > -static_cast<double>(__builtin_inff()) ? a + b : a;
}

// Whether the group `mine` of this lane, of the score `of_mine`, is taken; its
// lane `first` leaves the score in LDS. sure: rounding cannot have decided it,
// that is, too few groups may lie above it or enough certainly do.
template <typename S>
__device__ __forceinline__ bool taken(const ScoredArgs& p, S* score, int32_t mine, bool first, S of_mine,
                                      bool exact, bool& sure) {
  if (first && mine < p.groups) score[mine] = of_mine;
  wave_sync();
  const auto m = number(of_mine);
  int32_t before = 0, over = 0, near = 0;
#pragma unroll 4
  for (int32_t h = 0; h < p.groups; ++h) {
    const S s = score[h];
    before += number(s) > m || (number(s) == m && h < mine) ? 1 : 0;
    if constexpr (std::is_same<S, GroupScore>::value) {
      const float d = s.off + of_mine.off, t = s.v - m;
      over += t > d ? 1 : 0;
      near += h != mine && !(t < -d) ? 1 : 0;
    }
  }
  wave_sync();
  const bool open = m > -__builtin_inff();
  if (!exact && open && mine < p.groups && !(near < p.top_groups || over >= p.top_groups)) sure = false;
  return open && before < p.top_groups;
}

// The groups taken, as bits, of values in a row of LDS: a group by as many
// lanes as there are for all of them (more groups than lanes: several turns).
template <int G, typename T, typename S>
__device__ __forceinline__ uint64_t groups_of_row(const ScoredArgs& p, int32_t parts, const T* row, S* score,
                                                  int l, bool exact, float base, bool& sure) {
  const T none = -static_cast<T>(__builtin_inff());
  const int32_t turns = (p.groups * parts + G - 1) / G;
  for (int32_t i = 0; i < turns; ++i) {
    const int32_t g = (l + i * G) / parts, part = l % parts;
    T a = none, b = none;
    if (g < p.groups)
#pragma unroll 2
      for (int32_t z = part; z < p.group_size; z += parts) {
        const T t = row[g * p.group_size + z];
        b = t > a ? a : t > b ? t : b;
        a = t > a ? t : a;
      }
    butterfly<G>([&](auto step) {
      constexpr int kStep = decltype(step)::value;
      if (kStep < parts) join_two<kStep>(a, b);
    });
    if (g < p.groups && part == 0) score[g] = score_of(p, a, b, exact, base);
  }
  wave_sync();
  uint64_t bits = 0;
  for (int32_t i = 0; i * G < p.groups; ++i) {
    const int32_t g = l + i * G;
    const S of_mine = g < p.groups ? score[g] : score_of(p, none, none, true, 0.0f);
    const bool keep = taken(p, score, g, false, of_mine, exact, sure);
    const uint64_t all = __ballot(keep) >> ((threadIdx.x & 63) & ~(G - 1));
    bits |= (G == 64 ? all : all & ((1ull << (G & 63)) - 1)) << (i * G & 63);
  }
  return bits;
}

// Leaves only the values of the groups taken. A group of whole lanes, a power
// of two, is joined in registers, others through the row in LDS.
template <int G, int V>
__device__ __forceinline__ void keep_groups(const ScoredArgs& p, float (&v)[V], const float (&from)[V],
                                            float* row, GroupScore* score, int l, bool exact, float base,
                                            bool& sure) {
  const float none = -__builtin_inff();
  if (p.lanes_a_group != 0) {
    float a = none, b = none;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      b = __builtin_amdgcn_fmed3f(a, b, from[j]);
      a = from[j] > a ? from[j] : a;
    }
    butterfly<G>([&](auto step) {
      constexpr int kStep = decltype(step)::value;
      if (kStep < p.lanes_a_group) join_two<kStep>(a, b);
    });
    const int32_t mine = l / p.lanes_a_group;
    const bool keep = taken(p, score, mine, l % p.lanes_a_group == 0, score_of(p, a, b, exact, base), exact,
                            sure);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = keep ? v[j] : none;
    return;
  }
  const int32_t e0 = l * V;
#pragma unroll
  for (int j = 0; j < V; ++j) row[e0 + j] = from[j];
  wave_sync();
  const uint64_t bits = groups_of_row<G>(p, p.parts, row, score, l, exact, base, sure);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t g = static_cast<uint32_t>(e0 + j) / static_cast<uint32_t>(p.group_size);
    v[j] = g < 64u && ((bits >> g) & 1) ? v[j] : none;
  }
}

// A row's choice in fp64, by the whole wave: a lane has every 64th expert.
// Leaves the slots' experts in LDS.
template <int kExperts, bool kBf16>
__device__ __forceinline__ void settle(const ScoredArgs& p, int64_t row, float top, bool plain,
                                       bool exact_groups, double* values, double* score, int32_t* slots) {
  constexpr int kE = kExperts / 64;
  const int lane = threadIdx.x & 63;
  const int32_t n_experts = p.r.n_experts;
  const double nothing = -static_cast<double>(__builtin_inff());
  float x[kE];
  double v[kE], all = 0.0;
#pragma unroll
  for (int i = 0; i < kE; ++i) {
    const int32_t e = lane + 64 * i;
    x[i] = -__builtin_inff();
    if (e < n_experts)
      x[i] = kBf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p.r.logits)[row + e]) << 16)
                   : static_cast<const float*>(p.r.logits)[row + e];
    const double xv = x[i];
    v[i] = p.sigmoid ? (xv < 0.0 ? exp(xv) : 1.0) / (1.0 + exp(-fabs(xv)))
                     : exp(xv - static_cast<double>(top));
    all += v[i];
  }
  butterfly<64>([&](auto step) {
    uint64_t c, d;
    pair_of<decltype(step)::value>(__builtin_bit_cast(uint64_t, all), c, d);
    all = __builtin_bit_cast(double, c) + __builtin_bit_cast(double, d);
  });
  const bool grouped = p.groups > 1 && p.top_groups < p.groups;
#pragma unroll
  for (int i = 0; i < kE; ++i) {
    const int32_t e = lane + 64 * i;
    const bool open = x[i] > -__builtin_inff();
    const double bias = p.bias != nullptr && e < n_experts ? p.bias[e] : 0.0f;
    const double s = (p.sigmoid ? v[i] : v[i] / all) + bias;
    if (grouped) {
      const double g = exact_groups ? static_cast<double>(x[i]) : s;
      values[e] = open && g > nothing ? g : nothing;
    }
    v[i] = plain ? static_cast<double>(x[i]) : s;
    if (!open || !(v[i] > nothing)) v[i] = nothing;
  }
  if (grouped) {
    wave_sync();
    int32_t parts = 1;
    while (2 * parts * p.groups <= 64) parts *= 2;
    bool sure = true;
    const uint64_t bits = groups_of_row<64>(p, parts, values, score, lane, true, 0.0f, sure);
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const uint32_t g = static_cast<uint32_t>(lane + 64 * i) / static_cast<uint32_t>(p.group_size);
      v[i] = g < 64u && ((bits >> g) & 1) ? v[i] : nothing;
    }
  }
  for (int32_t n = 0; n < p.r.top_k; ++n) {
    double best = v[0];
    uint32_t at = lane;
#pragma unroll
    for (int i = 1; i < kE; ++i) {
      at = v[i] > best ? lane + 64 * i : at;
      best = v[i] > best ? v[i] : best;
    }
    butterfly<64>([&](auto step) {
      uint64_t c, d;
      uint32_t ac, ad;
      pair_of<decltype(step)::value>(__builtin_bit_cast(uint64_t, best), c, d);
      pair_of<decltype(step)::value>(at, ac, ad);
      const double bc = __builtin_bit_cast(double, c), bd = __builtin_bit_cast(double, d);
      const bool second = bd > bc || (bd == bc && ad < ac);
      best = second ? bd : bc;
      at = second ? ad : ac;
    });
#pragma unroll
    for (int i = 0; i < kE; ++i) v[i] = at == static_cast<uint32_t>(lane + 64 * i) ? nothing : v[i];
    if (lane == 0) slots[n] = best > nothing ? static_cast<int32_t>(at) : -1;
  }
}

template <int G, int V, bool kBf16, bool kSort>
__global__ __launch_bounds__(64 * kWavesABlock) void scored_kernel(ScoredArgs a) {
  constexpr int kRows = 64 / G, kExperts = G * V;
  constexpr int kHeld = kSort ? 1 : kMaxTopK / G;
  __shared__ int32_t counts[kExperts + 1];
  __shared__ double red[kWavesABlock];
  // a row's logits and values; in fp64, values over both
  __shared__ __align__(16) double row_s[kWavesABlock][kRows][kExperts];
  __shared__ double g_s[kWavesABlock][kRows][kMaxGroups];
  __shared__ int32_t slot_s[kWavesABlock][kRows][kSort ? kSorted : kMaxTopK];
  const RouteArgs& p = a.r;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & (G - 1), mine = lane / G;
  const int32_t e0 = l * V;
  const bool stats = p.counts != nullptr;
  if (stats) {
    for (int32_t e = threadIdx.x; e <= p.n_experts; e += blockDim.x) counts[e] = 0;
    __syncthreads();
  }
  const bool grouped = a.groups > 1 && a.top_groups < a.groups;
  float bias[V], sums[V];
  bool zero = true, number = true;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    bias[j] = a.bias != nullptr && e0 + j < p.n_experts ? a.bias[e0 + j] : 0.0f;
    zero &= bias[j] == 0.0f;
    number &= bias[j] == bias[j];
    sums[j] = 0.0f;
  }
  // a bias of zeros is none
  const bool by_logit = __ballot(!zero) == 0;
  const bool nan_bias = __ballot(!number) != 0;
  double* d_row = row_s[wave][mine];
  float* x_row = reinterpret_cast<float*>(d_row);
  float* v_row = x_row + kExperts;
  GroupScore* g_row = reinterpret_cast<GroupScore*>(g_s[wave][mine]);
  int32_t* slot_row = slot_s[wave][mine];
  const float none = -__builtin_inff();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWavesABlock * kRows;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWavesABlock + wave) * kRows; t0 < p.n_tokens;
       t0 += step) {
    const int64_t t = t0 + mine;
    const bool in = t < p.n_tokens;
    const bool valid = in && (p.valid == nullptr || p.valid[t] != 0);
    Logits<V, kBf16> x;
    x.load(p.logits, (in ? t : t0) * p.ld, e0, p.n_experts, p.vec);
    float top = x.value(0), low = top;
#pragma unroll
    for (int j = 1; j < V; ++j) {
      top = fmaxf(top, x.value(j));
      low = fminf(low, x.value(j));
    }
    top = group_max<G>(top);
    // scores relative to exp(shift), and their sum
    const float shift = a.sigmoid ? fminf(top, 0.0f) : top;
    float s[V], total = 0.0f;
    if (!a.sigmoid) {
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] = exp_of(x.value(j) - top);
    } else if (__ballot(shift < 0.0f) == 0) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xv = x.value(j), e = low_exp(xv);
        s[j] = (xv >= 0.0f ? 1.0f : e) * inverse(1.0f + e);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xv = x.value(j);
        s[j] = (xv >= 0.0f ? 1.0f : exp_of(xv - shift)) * inverse(1.0f + low_exp(xv));
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) total += s[j];
#pragma unroll
    for (int j = 0; j < V; j += 4)
      *reinterpret_cast<float4*>(x_row + e0 + j) =
          float4{x.value(j), x.value(j + 1), x.value(j + 2), x.value(j + 3)};
    total = group_sum<G>(total);
    const float inv = inverse(total);
    // what is compared
    const bool no_numbers = !a.sigmoid && total != total, plain = by_logit || no_numbers;
    const bool exact_groups = plain && (a.group_best == 1 || no_numbers);
    const float base = a.sigmoid ? kSigmoidBase : kSoftmaxBase * inv;
    const float whole = a.sigmoid ? (shift < 0.0f ? exp_of(shift) : 1.0f) : inv;
    float v[V];
    bool sure = true;
    // closed experts, or no numbers: each value looked at (a NaN's key would lie
    // above all others)
    const bool special = nan_bias || __ballot(!(low > none) || total != total) != 0;
    if (special || by_logit) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xv = x.value(j), w = plain ? xv + 0.0f : __builtin_fmaf(s[j], whole, bias[j]);
        v[j] = xv > none && w > none ? w : none;
      }
      if (grouped) {
        float from[V];
#pragma unroll
        for (int j = 0; j < V; ++j)
          from[j] = exact_groups || !(v[j] > none) ? v[j] : __builtin_fmaf(s[j], whole, bias[j]);
        keep_groups<G, V>(a, v, from, v_row, g_row, l, exact_groups, base, sure);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = __builtin_fmaf(s[j], whole, bias[j]);
      if (grouped) keep_groups<G, V>(a, v, v, v_row, g_row, l, false, base, sure);
    }
    // lane l of the row: slots l, l + G, ..; -1 where none is left
    int32_t slot[kHeld];
    const bool keyed = kBf16 && kSort && __ballot(!plain) == 0;   // the expert is in the key
    if constexpr (kSort) {
      slot[0] = -1;
      if (keyed) {
        uint32_t key[V], best[8];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const uint32_t o = order_of(v[j]);
          key[j] = o == 0 ? 0u : (o & 0xFFFF0000u) | (0xFFFFu - static_cast<uint32_t>(e0 + j));
        }
        best8<G, V>(key, best);
#pragma unroll
        for (int j = 0; j < kSorted; ++j)
          if (l == j && best[j] != 0) slot[0] = static_cast<int32_t>(0xFFFFu - (best[j] & 0xFFFFu));
      } else {
        int32_t key[V], best[8];
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = ordered(v[j]);
        best8<G, V>(key, best);
        // gaps between the slots and to the best left out
        const float first = fabsf(value_of(best[0]));
        int32_t last = best[0];
        uint32_t filled = best[0] > kNone ? 1u : 0u;
#pragma unroll
        for (int j = 1; j < kSorted; ++j) {
          if (j >= p.top_k) break;
          last = best[j];
          const float b = value_of(best[j]), gap = value_of(best[j - 1]) - b;
          if (best[j] > kNone) {
            sure &= plain ? gap > 0.0f : gap > apart(base, fmaxf(fabsf(b), first));
            ++filled;
          }
        }
        int32_t next = kNone;
        uint32_t own = 0;   // this lane's experts among the slots
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int32_t left = key[j] < last ? key[j] : kNone;
          next = left > next ? left : next;
          own |= key[j] >= last ? 1u << j : 0u;
        }
        if (last == kNone) {
          own = 0;
#pragma unroll
          for (int j = 0; j < V; ++j) own |= key[j] > kNone ? 1u << j : 0u;
        }
        next = group_max_key<G>(next);
        if (last > kNone && next > kNone && !plain) {
          const float b = value_of(next);
          sure &= value_of(last) - b > apart(base, fmaxf(fabsf(b), first));
        }
        // equal values at the end of the slots: more experts than slots
        sure &= group_sum<G>(static_cast<float>(__builtin_popcount(own))) == static_cast<float>(filled);
        if (l < kSorted) slot_row[l] = -1;
#pragma unroll
        for (int j = 0; j < V; j += 4)
          *reinterpret_cast<int4*>(reinterpret_cast<int32_t*>(v_row) + e0 + j) =
              int4{key[j], key[j + 1], key[j + 2], key[j + 3]};
        wave_sync();
        while (own != 0) {
          const int j = __builtin_ctz(own);
          own &= own - 1;
          const int32_t k = reinterpret_cast<const int32_t*>(v_row)[e0 + j];
          int32_t n = 0;
#pragma unroll
          for (int q = 0; q < kSorted; ++q) n += best[q] > k ? 1 : 0;
          if (n < kSorted) slot_row[n] = e0 + j;
        }
        wave_sync();
        if (l < kSorted) slot[0] = slot_row[l];
      }
    } else {
      uint64_t key[V], last = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t o = order_of(v[j]);
        key[j] = o == 0 ? 0u : (static_cast<uint64_t>(o) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(e0 + j));
      }
      int32_t n = 0;
      float first = 0.0f, before = 0.0f;
#pragma unroll
      for (int h = 0; h < kHeld; ++h) {
        slot[h] = -1;
        for (int j = 0; j < G && n <= p.top_k; ++j, ++n) {   // one more: the best left out
          last = key[0];
#pragma unroll
          for (int q = 1; q < V; ++q) last = key[q] > last ? key[q] : last;
          last = group_max_key<G>(last);
#pragma unroll
          for (int q = 0; q < V; ++q) key[q] = key[q] == last ? 0 : key[q];
          if (l == j && last != 0 && n < p.top_k) slot[h] = KeyF32::expert(last);
          const float b = KeyF32::value(last);
          if (n == 0) first = b;
          if (!plain && n > 0 && last != 0) sure &= before - b > apart(base, fmaxf(fabsf(b), fabsf(first)));
          before = b;
        }
      }
      // 64 slots leave no turn for the best left out
      if (!plain && n <= p.top_k && last != 0) sure = false;
    }
    const uint64_t unsettled = __ballot(!sure && valid);
    if (unsettled != 0) {   // rare: these rows in fp64
      wave_sync();
#pragma unroll 1
      for (int row = 0; row < kRows; ++row) {
        const int at = row * G;
        if (((unsettled >> at) & (G == 64 ? ~0ull : (1ull << (G & 63)) - 1)) == 0) continue;
        settle<kExperts, kBf16>(a, (t0 + row) * p.ld, __shfl(top, at, 64), __shfl(plain ? 1 : 0, at, 64) != 0,
                                __shfl(exact_groups ? 1 : 0, at, 64) != 0, row_s[wave][row], g_s[wave][row],
                                slot_s[wave][row]);
        wave_sync();
        if (mine == row) {
#pragma unroll
          for (int h = 0; h < kHeld; ++h)
            slot[h] = l + h * G < p.top_k ? slot_row[l + h * G] : -1;
        }
      }
      wave_sync();
#pragma unroll
      for (int j = 0; j < V; ++j) x_row[e0 + j] = x.value(j);
      wave_sync();
    }
    // weights of the slots
    float e[kHeld], xs[kHeld], high = none, taken = 0.0f;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      if (l + h * G >= p.top_k) slot[h] = -1;
      xs[h] = slot[h] >= 0 ? x_row[slot[h]] : none;
      high = fmaxf(high, xs[h]);
    }
    high = group_max<G>(high);
    const bool counted = valid && high > none;
    const float from = !p.renorm ? (a.sigmoid ? 0.0f : top) : a.sigmoid ? fminf(high, 0.0f) : high;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      e[h] = 0.0f;
      if (slot[h] >= 0)
        e[h] = a.sigmoid ? exp_of(fminf(xs[h], 0.0f) - from) * inverse(1.0f + low_exp(xs[h]))
                         : exp_of(xs[h] - from);
      taken += e[h];
    }
    if (p.renorm) taken = group_sum<G>(taken);
    // a NaN among the logits is one of every softmax weight
    const float f = no_numbers ? total : p.renorm ? inverse(taken) : a.sigmoid ? 1.0f : inv;
    if (stats) {
      if (__ballot(!counted) == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) sums[j] = __builtin_fmaf(s[j], inv, sums[j]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) sums[j] = counted ? __builtin_fmaf(s[j], inv, sums[j]) : sums[j];
      }
      if (counted && l == 0) atomicAdd(&counts[p.n_experts], 1);
    }
    if (in) {
#pragma unroll
      for (int h = 0; h < kHeld; ++h) {
        const int32_t n = l + h * G;
        if ((kSort && l >= kSorted) || n >= p.top_k) continue;
        const bool some = counted && slot[h] >= 0;
        p.idx[t * p.top_k + n] = some ? slot[h] : -1;
        p.weights[t * p.top_k + n] = some ? e[h] * f * a.scale : 0.0f;
        if (stats && some) atomicAdd(&counts[slot[h]], 1);
      }
    }
    wave_sync();
  }
  if (!stats) return;
  __syncthreads();
  // the wave's rows, then the block's waves, in a fixed order
  float(*prob)[kExperts] = reinterpret_cast<float(*)[kExperts]>(&row_s[0][0][0]);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float s = sums[j];
    uint32_t b, c;
    if (G <= 8) s += __shfl_xor(s, 8, 64);
    if (G <= 16) {
      pair_of<16>(__float_as_uint(s), b, c);
      s = __uint_as_float(b) + __uint_as_float(c);
    }
    if (G <= 32) {
      pair_of<32>(__float_as_uint(s), b, c);
      s = __uint_as_float(b) + __uint_as_float(c);
    }
    if (lane < G) prob[wave][e0 + j] = s;
  }
  __syncthreads();
  const bool alone = gridDim.x == 1;
  double term = 0.0;
  for (int32_t e = threadIdx.x; e <= p.n_experts; e += blockDim.x) {
    (alone ? p.counts : p.part_counts + static_cast<int64_t>(blockIdx.x) * (p.n_experts + 1))[e] =
        counts[e];
    if (e == p.n_experts) continue;
    double s = 0.0;
    for (int w = 0; w < kWavesABlock; ++w) s += prob[w][e];
    (alone ? p.prob_sum : p.part_prob + static_cast<int64_t>(blockIdx.x) * p.n_experts)[e] =
        static_cast<float>(s);
    term += counts[e] * s;
  }
  if (alone) {
    term = block_sum(term, red);
    if (threadIdx.x == 0) p.loss[0] = loss_of(term, p.n_experts, p.top_k, counts[p.n_experts]);
  } else if (blockIdx.x == 0 && threadIdx.x == 0) {
    *p.ticket = 0;
  }
}

// ---------------------------------------------------------------- backward
struct ScoredGradArgs {
  const void* logits;
  const int32_t* idx;
  const float* dweights;
  const int32_t* counts;
  const float* dloss;
  void* dlogits;
  uint32_t* status;
  int64_t ld, ld_d, n_tokens;
  int32_t n_experts, top_k;
  float scale;
  bool renorm, sigmoid, vec, vec_d;
};

// With t[e] the slots' scores over their sum (renormalised) and q[e] all
// scores over theirs, u and h the sums of dweights and the number of an
// expert's slots and f the loss's share: the weights give t (u - h sum u t) or
// s u, the loss q (f - sum f q), each times 1 - s for a sigmoid; a softmax that
// is not renormalised p (u - sum u p). The slots' gradients reach their
// experts' lanes through rows of LDS, as in moe_route.hip. 65536 rows of 256
// experts: 43 us for 138 MB, 27 of them at a copy's rate.
template <int G, int V, bool kBf16, bool kOutBf16>
__global__ __launch_bounds__(256) void scored_grad_kernel(ScoredGradArgs p) {
  constexpr int kRows = 64 / G, kExperts = G * V, kHeld = kMaxTopK / G;
  __shared__ __align__(16) float grad_s[4 * kRows][kExperts];
  __shared__ __align__(16) float hits_s[4 * kRows][kExperts];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & (G - 1);
  const int32_t e0 = l * V;
  float* grad_row = grad_s[wave * kRows + lane / G];
  float* hits_row = hits_s[wave * kRows + lane / G];
  constexpr int kPieces = V / 4;
  const auto place = [](int32_t e) {   // of expert e in a row
    const int32_t of = e / V, piece = e / 4 % kPieces;
    return of * V + 4 * (piece ^ ((of >> 2) & (kPieces - 1))) + e % 4;
  };
#pragma unroll
  for (int j = 0; j < V; ++j) grad_row[e0 + j] = hits_row[e0 + j] = 0.0f;
  wave_sync();
  float load[V];
#pragma unroll
  for (int j = 0; j < V; ++j) load[j] = 0.0f;
  const bool balance = p.counts != nullptr;
  if (balance) {
    const int32_t r = p.counts[p.n_experts];
    const float rows = static_cast<float>(r > 0 ? r : 1);
    const float f = p.dloss[0] * static_cast<float>(p.n_experts) /
                    (static_cast<float>(p.top_k) * rows) / rows;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (e0 + j < p.n_experts) load[j] = f * static_cast<float>(p.counts[e0 + j]);
  }
  const float none = -__builtin_inff();
  const int64_t step = static_cast<int64_t>(gridDim.x) * 4 * kRows;
  Logits<V, kBf16> next;
  int32_t e_next[kHeld];
  float w_next[kHeld];
  const auto request = [&](int64_t t0) __attribute__((always_inline)) {
    const int64_t t = t0 + lane / G;
    const bool in = t < p.n_tokens;
    const int64_t row = in ? t : p.n_tokens - 1;
    next.load(p.logits, row * p.ld, e0, p.n_experts, p.vec);
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      if (h * G >= p.top_k) break;
      const int32_t s = l + h * G;
      const int64_t at = row * p.top_k + (s < p.top_k ? s : 0);
      e_next[h] = p.idx[at];
      w_next[h] = p.dweights != nullptr ? p.dweights[at] : 0.0f;
      if (!in || s >= p.top_k) e_next[h] = -1;
    }
  };
  int64_t t0 = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * kRows;
  if (t0 >= p.n_tokens) return;
  request(t0);
  for (; t0 < p.n_tokens; t0 += step) {
    const int64_t t = t0 + lane / G;
    const Logits<V, kBf16> x = next;
    int32_t e[kHeld];
    bool counted = false;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      if (h * G >= p.top_k) break;
      e[h] = e_next[h];
      if (e[h] < 0 || e[h] >= p.n_experts) {
        if (e[h] != -1 && p.status != nullptr)
          atomicOr(p.status, static_cast<uint32_t>(BINADE_DEV_BAD_INDEX));
        e[h] = -1;
        continue;
      }
      counted |= h == 0 && l == 0;
      atomicAdd(&hits_row[place(e[h])], 1.0f);
      if (p.dweights != nullptr) atomicAdd(&grad_row[place(e[h])], w_next[h]);
    }
    if (t0 + step < p.n_tokens) request(t0 + step);
    wave_sync();
    counted = (__ballot(counted) >> (lane & ~(G - 1)) & 1u) != 0;
    float u[V], hits[V];
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      __builtin_memcpy(&u[4 * q], &grad_row[place(e0 + 4 * q)], 16);
      __builtin_memcpy(&hits[4 * q], &hits_row[place(e0 + 4 * q)], 16);
    }
    float top = x.value(0), high = none;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      top = fmaxf(top, x.value(j));
      high = hits[j] != 0.0f ? fmaxf(high, x.value(j)) : high;
    }
    top = group_max<G>(top);
    high = group_max<G>(high);
    float d[V];
    // scores over their sum q; for a sigmoid also s itself and 1 - s
    float q[V], s[V], rest[V], total = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float xv = x.value(j);
      if (p.sigmoid) {
        const float ex = low_exp(xv), in = inverse(1.0f + ex);
        s[j] = xv >= 0.0f ? in : ex * in;
        rest[j] = xv >= 0.0f ? ex * in : in;
        q[j] = exp_of(fminf(xv, 0.0f) - fminf(top, 0.0f)) * in;
      } else {
        q[j] = exp_of(xv - top);
        rest[j] = 1.0f;
      }
      total += q[j];
    }
    const float inv = inverse(group_sum<G>(total));
    float mean = 0.0f, shares = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      q[j] *= inv;
      shares = __builtin_fmaf(q[j], load[j], shares);
    }
    if (p.renorm) {
      float tv[V], sum = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xv = x.value(j);
        tv[j] = 0.0f;
        if (hits[j] != 0.0f)
          tv[j] = p.sigmoid ? exp_of(fminf(xv, 0.0f) - fminf(high, 0.0f)) * inverse(1.0f + low_exp(xv))
                            : exp_of(xv - high);
        sum = __builtin_fmaf(hits[j], tv[j], sum);
        mean = __builtin_fmaf(u[j], tv[j], mean);
      }
      const float f = inverse(group_sum<G>(sum));
      mean = group_sum<G>(mean) * f;
#pragma unroll
      for (int j = 0; j < V; ++j) d[j] = p.scale * (tv[j] * f) * (u[j] - hits[j] * mean);
    } else if (p.sigmoid) {
#pragma unroll
      for (int j = 0; j < V; ++j) d[j] = u[j] != 0.0f ? p.scale * s[j] * u[j] : 0.0f;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) mean = __builtin_fmaf(q[j], u[j], mean);
      mean = group_sum<G>(mean);
#pragma unroll
      for (int j = 0; j < V; ++j) d[j] = p.scale * q[j] * (u[j] - mean);
    }
    if (balance) {
      shares = group_sum<G>(shares);
#pragma unroll
      for (int j = 0; j < V; ++j) d[j] = __builtin_fmaf(q[j], load[j] - shares, d[j]);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = counted ? d[j] * rest[j] : 0.0f;
    wave_sync();
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      if (h * G >= p.top_k) break;
      if (e[h] >= 0) grad_row[place(e[h])] = hits_row[place(e[h])] = 0.0f;
    }
    wave_sync();
    if (t >= p.n_tokens) continue;
    const int64_t row = t * p.ld_d;
#pragma unroll
    for (int b = 0; b < V / 8; ++b) {
      const int32_t ex = e0 + 8 * b;
      if (p.vec_d) {
        if (ex >= p.n_experts) continue;
        if (kOutBf16) {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = pack_bf16(d[8 * b + 2 * j], d[8 * b + 2 * j + 1]);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dlogits) + row + ex) =
              uint4{o[0], o[1], o[2], o[3]};
        } else {
          __builtin_memcpy(__builtin_assume_aligned(static_cast<float*>(p.dlogits) + row + ex, 16),
                           &d[8 * b], 32);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (ex + j >= p.n_experts) continue;
          if (kOutBf16) static_cast<uint16_t*>(p.dlogits)[row + ex + j] = to_bf16_rne(d[8 * b + j]);
          else static_cast<float*>(p.dlogits)[row + ex + j] = d[8 * b + j];
        }
      }
    }
  }
}

// ------------------------------------------------------------------- hosts
// Experts a lane, and lanes a row. With few tokens the chain of one row's
// instructions counts, and eight experts a lane make it shorter; with many
// their number does: sixteen (more than 512 experts take a whole wave's). 8 of
// 256 experts in groups, in a graph, us with eight and with sixteen, fp32 logits
// (bf16), of eight sets of logits the least:
//   512 tokens 7.9 and 9.9 (8.0, 10.1)     1024: 8.0 and 10.0 (8.2, 10.1)
//   2048: 8.1 and 10.1 (8.3, 10.2)         4096: 10.2 and 10.3 (13.7, 15.7)
//   16384: 29.8 and 24.7 (29.7, 32.9)
// With counts 1024: 14.2 and 15.7 (14.1, 15.8); of 512 experts with counts 1024:
// 15.9 and 17.9 (15.8, 17.6), 2048: 21.4 and 18.6 (21.5, 18.6). So 1024 is where
// eight are still faster for every number of experts. A row that fp32 does not
// settle adds 6 us to any of these: one in a few thousand here.
constexpr int64_t kFewTokens = 1024;
int32_t scored_each(int64_t n_tokens, int32_t n_experts) {
  return n_experts <= 64 || (n_experts <= 512 && n_tokens <= kFewTokens) ? 8 : 16;
}
int32_t scored_lanes(int64_t n_tokens, int32_t n_experts) {
  const int32_t held = 8 * scored_each(n_tokens, n_experts);   // of the fewest lanes
  return n_experts <= held ? 8 : n_experts <= 2 * held ? 16 : n_experts <= 4 * held ? 32 : 64;
}

uint32_t scored_blocks(int64_t n_tokens, int32_t n_experts) {
  const int64_t rows = kWavesABlock * (64 / scored_lanes(n_tokens, n_experts));
  const int64_t b = (n_tokens + rows - 1) / rows;
  return static_cast<uint32_t>(b < 1 ? 1 : b > kScoredBlocks ? kScoredBlocks : b);
}

template <int G, int V>
void launch_scored(const ScoredArgs& p, uint32_t blocks, bool bf16, hipStream_t st) {
  const dim3 grid(blocks), block(64 * kWavesABlock);
  const bool sort = p.r.top_k <= kSorted;
  if (bf16 && sort) hipLaunchKernelGGL((scored_kernel<G, V, true, true>), grid, block, 0, st, p);
  else if (bf16) hipLaunchKernelGGL((scored_kernel<G, V, true, false>), grid, block, 0, st, p);
  else if (sort) hipLaunchKernelGGL((scored_kernel<G, V, false, true>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((scored_kernel<G, V, false, false>), grid, block, 0, st, p);
}

template <int G, int V>
void launch_scored_grad(const ScoredGradArgs& p, bool bf16, bool out_bf16, hipStream_t st) {
  const int64_t rows = 4 * (64 / G), b = (p.n_tokens + rows - 1) / rows;
  const dim3 grid(static_cast<uint32_t>(b < 1024 ? b : 1024)), block(256);
  if (bf16 && out_bf16) hipLaunchKernelGGL((scored_grad_kernel<G, V, true, true>), grid, block, 0, st, p);
  else if (bf16) hipLaunchKernelGGL((scored_grad_kernel<G, V, true, false>), grid, block, 0, st, p);
  else if (out_bf16) hipLaunchKernelGGL((scored_grad_kernel<G, V, false, true>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((scored_grad_kernel<G, V, false, false>), grid, block, 0, st, p);
}

bool score_ok(int32_t score) { return score == BINADE_SOFTMAX || score == BINADE_SIGMOID; }

}  // namespace
}  // namespace binade

using namespace binade;

extern "C" int64_t binade_moe_route_scored_workspace_bytes(int64_t n_tokens, int32_t n_experts) {
  if (!route_sizes_ok(n_tokens, n_experts)) return 0;
  // up to kFewTokens there may be more blocks than for a few tokens more
  const int64_t few = n_tokens < kFewTokens ? n_tokens : kFewTokens;
  const int64_t a = scored_blocks(n_tokens, n_experts), b = scored_blocks(few, n_experts);
  return kHead + (a > b ? a : b) * (2 * n_experts + 1) * 4;
}

extern "C" int32_t binade_moe_route_scored(const void* logits, int32_t dtype, int64_t ld,
                                           int64_t n_tokens, int32_t n_experts, int32_t top_k,
                                           const binade_route_rule* rule, const uint8_t* valid,
                                           int32_t* idx, float* weights, int32_t* counts,
                                           float* prob_sum, float* loss, void* workspace,
                                           int64_t workspace_bytes, void* stream) {
  if (!route_sizes_ok(n_tokens, n_experts) || top_k < 1 || top_k > n_experts || top_k > kMaxTopK ||
      ld < n_experts || rule == nullptr)
    return BINADE_EINVAL;
  if (dtype != BINADE_F32 && dtype != BINADE_BF16) return BINADE_EINVAL;
  if (!score_ok(rule->score) || rule->groups < 1 || rule->groups > kMaxGroups ||
      n_experts % rule->groups != 0 || rule->top_groups < 1 || rule->top_groups > rule->groups ||
      (rule->group_best != 1 && rule->group_best != 2) ||
      top_k > rule->top_groups * (n_experts / rule->groups) || !__builtin_isfinite(rule->scale))
    return BINADE_EINVAL;
  const bool stats = counts != nullptr;
  if (stats != (prob_sum != nullptr) || stats != (loss != nullptr)) return BINADE_EINVAL;
  if (n_tokens == 0 && !stats) return BINADE_OK;
  if (n_tokens > 0 && (logits == nullptr || idx == nullptr || weights == nullptr))
    return BINADE_EINVAL;
  if (stats) {
    if (workspace == nullptr ||
        workspace_bytes < binade_moe_route_scored_workspace_bytes(n_tokens, n_experts))
      return BINADE_ENOSPACE;
    if (!aligned16(workspace)) return BINADE_EUNSUPPORTED;
  }
  const uint32_t blocks = scored_blocks(n_tokens, n_experts);
  ScoredArgs a{};
  RouteArgs& p = a.r;
  p.logits = logits;
  p.valid = valid;
  p.idx = idx;
  p.weights = weights;
  p.counts = counts;
  p.prob_sum = prob_sum;
  p.loss = loss;
  p.ticket = static_cast<uint32_t*>(workspace);
  p.part_loss = static_cast<double*>(workspace) + 8;
  p.part_counts = static_cast<int32_t*>(workspace) + kHead / 4;
  p.part_prob = reinterpret_cast<float*>(p.part_counts + static_cast<int64_t>(blocks) * (n_experts + 1));
  p.ld = ld;
  p.n_tokens = n_tokens;
  p.n_experts = n_experts;
  p.top_k = top_k;
  p.renorm = rule->renormalize != 0;
  const bool bf16 = dtype == BINADE_BF16;
  p.vec = whole_pieces(logits, n_experts, ld, bf16);
  a.bias = rule->bias;
  a.groups = rule->groups;
  a.group_size = n_experts / rule->groups;
  a.top_groups = rule->top_groups;
  a.group_best = rule->group_best;
  const int32_t lanes = scored_lanes(n_tokens, n_experts), each = scored_each(n_tokens, n_experts);
  const int32_t whole = a.group_size % each == 0 ? a.group_size / each : 0;
  a.lanes_a_group = (whole & (whole - 1)) == 0 ? whole : 0;
  a.parts = 1;
  while (2 * a.parts * a.groups <= lanes) a.parts *= 2;
  a.scale = rule->scale;
  a.sigmoid = rule->score == BINADE_SIGMOID;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (each == 8) {
    if (lanes == 8) launch_scored<8, 8>(a, blocks, bf16, st);
    else if (lanes == 16) launch_scored<16, 8>(a, blocks, bf16, st);
    else if (lanes == 32) launch_scored<32, 8>(a, blocks, bf16, st);
    else launch_scored<64, 8>(a, blocks, bf16, st);
  } else {
    if (lanes == 8) launch_scored<8, 16>(a, blocks, bf16, st);
    else if (lanes == 16) launch_scored<16, 16>(a, blocks, bf16, st);
    else if (lanes == 32) launch_scored<32, 16>(a, blocks, bf16, st);
    else launch_scored<64, 16>(a, blocks, bf16, st);
  }
  if (stats && blocks > 1)
    hipLaunchKernelGGL(route_stats_kernel, dim3(static_cast<uint32_t>((n_experts + 63) / 64)),
                       dim3(1024), 0, st, p, static_cast<int32_t>(blocks));
  return launch_status();
}

extern "C" int32_t binade_moe_route_scored_grad(const void* logits, int32_t dtype, int64_t ld,
                                                int64_t n_tokens, int32_t n_experts, int32_t top_k,
                                                int32_t score, int32_t renormalize, float scale,
                                                const int32_t* idx, const float* dweights,
                                                const int32_t* counts, const float* dloss,
                                                void* dlogits, int32_t dlogits_dtype, int64_t ld_d,
                                                uint32_t* dev_status, void* stream) {
  if (!route_sizes_ok(n_tokens, n_experts) || top_k < 1 || top_k > n_experts || top_k > kMaxTopK ||
      ld < n_experts || ld_d < n_experts || !score_ok(score) || !__builtin_isfinite(scale))
    return BINADE_EINVAL;
  if ((dtype != BINADE_F32 && dtype != BINADE_BF16) ||
      (dlogits_dtype != BINADE_F32 && dlogits_dtype != BINADE_BF16))
    return BINADE_EINVAL;
  if ((counts != nullptr) != (dloss != nullptr)) return BINADE_EINVAL;
  if (n_tokens == 0) return BINADE_OK;
  if (logits == nullptr || idx == nullptr || dlogits == nullptr) return BINADE_EINVAL;
  const bool bf16 = dtype == BINADE_BF16, out_bf16 = dlogits_dtype == BINADE_BF16;
  ScoredGradArgs p{};
  p.logits = logits;
  p.idx = idx;
  p.dweights = dweights;
  p.counts = counts;
  p.dloss = dloss;
  p.dlogits = dlogits;
  p.status = dev_status;
  p.ld = ld;
  p.ld_d = ld_d;
  p.n_tokens = n_tokens;
  p.n_experts = n_experts;
  p.top_k = top_k;
  p.scale = scale;
  p.renorm = renormalize != 0;
  p.sigmoid = score == BINADE_SIGMOID;
  p.vec = whole_pieces(logits, n_experts, ld, bf16);
  p.vec_d = whole_pieces(dlogits, n_experts, ld_d, out_bf16);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (n_experts <= 64) launch_scored_grad<8, 8>(p, bf16, out_bf16, st);
  else if (n_experts <= 128) launch_scored_grad<16, 8>(p, bf16, out_bf16, st);
  else if (n_experts <= 256) launch_scored_grad<32, 8>(p, bf16, out_bf16, st);
  else if (n_experts <= 512) launch_scored_grad<64, 8>(p, bf16, out_bf16, st);
  else launch_scored_grad<64, 16>(p, bf16, out_bf16, st);
  return launch_status();
}
