// The router of a MoE layer and its backward: softmax, top-k, per-expert
// counts, balance loss (the arithmetic is stated in binade.h).
//
// A row belongs to a group of G lanes with V adjacent experts each (64, 128,
// 256, 512 or 1024 in all), so a wave has 64 / G rows at once: what a row
// costs is instructions, not bytes, and a lane's own sort is cheaper than
// steps across lanes. 16 experts a lane for bf16; 8 for fp32, whose keys take
// two registers each (with 16 they spill). Nothing of a row leaves its group;
// sums over rows stay in the lanes' registers (a lane's experts never change)
// until the block ends.
//
// Choice. A logit and its expert make one whole-number key (bf16: 16 + 16
// bits, fp32: 32 + 32), larger for the larger logit and, among equal ones,
// for the smaller expert, so that max and min alone sort. For top_k <= 8 each
// lane sorts its keys by a network, and log2 G steps merge a lane's best
// eight with its partner's (max(a[j], b[7 - j]) keeps the best eight of two
// sorted lists). For more slots the best key is taken out top_k times.
#include "moe_route.h"

namespace binade {
namespace {

constexpr int32_t kBlocks = 256;  // at most: each leaves one row of partial sums

// ----------------------------------------------------------------- forward
// Measured: 65536 tokens of 256 bf16 experts, top 8, counts and sums, 22.1 us
// (7 us of bytes): 563 vector instructions a wave's four rows, most of them
// the keys' sorting and the merge's four steps, 15 us at the issue rate; 2048
// tokens of 128 fp32 experts 5.8, one token 2.5. Both kernels in a captured
// graph 27.3 us for 8 slots of the first, 33.9 for 10, 41 for 16, 110 for 64.
template <int G, int V, typename K, bool kSort>
__global__ __launch_bounds__(1024) void route_kernel(RouteArgs p) {
  typedef typename K::Key Key;
  constexpr bool kBf16 = sizeof(Key) == 4;
  constexpr int kRows = 64 / G;           // of a wave
  constexpr int kExperts = G * V;
  __shared__ int32_t counts[kExperts + 1];
  __shared__ float prob[16][kExperts];
  __shared__ double red[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int l = lane & (G - 1);
  const int32_t e0 = l * V;
  const bool stats = p.counts != nullptr;
  if (stats) {
    for (int32_t e = threadIdx.x; e <= p.n_experts; e += blockDim.x) counts[e] = 0;
    __syncthreads();
  }
  float sums[V];
#pragma unroll
  for (int j = 0; j < V; ++j) sums[j] = 0.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * waves * kRows;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * waves + wave) * kRows; t0 < p.n_tokens;
       t0 += step) {
    const int64_t t = t0 + lane / G;
    const bool in = t < p.n_tokens;
    const bool valid = in && (p.valid == nullptr || p.valid[t] != 0);
    Logits<V, kBf16> x;
    x.load(p.logits, (in ? t : t0) * p.ld, e0, p.n_experts, p.vec);
    Key key[V], best[8];
    const auto choose = [&]() __attribute__((always_inline)) {
      if (kSort) {
        best8<G, V>(key, best);
      } else {
        best[0] = key[0];
#pragma unroll
        for (int j = 1; j < V; ++j) best[0] = key[j] > best[0] ? key[j] : best[0];
        best[0] = group_max_key<G>(best[0]);
      }
    };
    K::template make<V, false>(x, e0, key);
    choose();
    // NaN above +inf is rare: seen by the best key, and left out then
    if (__ballot(K::order_of(best[0]) > K::kHigh) != 0) {
      K::template make<V, true>(x, e0, key);
      choose();
    }
    const bool counted = valid && K::order_of(best[0]) > K::kLow;
    const float top = K::value(best[0]);
    float v[V], total = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v[j] = exp_of(x.value(j) - top);
      total += v[j];
    }
    total = group_sum<G>(total);
    const float inv = inverse(total);
    if (stats) {
      if (__ballot(!counted) == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) sums[j] = __builtin_fmaf(v[j], inv, sums[j]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) sums[j] = counted ? __builtin_fmaf(v[j], inv, sums[j]) : sums[j];
      }
      if (counted && l == 0) atomicAdd(&counts[p.n_experts], 1);
    }
    // lane l of the group: slots l, l + G, ... of the row
    constexpr int kHeld = kSort ? 1 : kMaxTopK / G > 0 ? kMaxTopK / G : 1;
    Key slot[kHeld];
    if (kSort) {
      slot[0] = best[0];
#pragma unroll
      for (int j = 1; j < kSorted; ++j) slot[0] = l == j ? best[j] : slot[0];
    } else {
      int32_t s = 0;
#pragma unroll
      for (int h = 0; h < kHeld; ++h) {
        slot[h] = 0;
        for (int j = 0; j < G && s < p.top_k; ++j, ++s) {
          if (s > 0) {
            best[0] = key[0];
#pragma unroll
            for (int q = 1; q < V; ++q) best[0] = key[q] > best[0] ? key[q] : best[0];
            best[0] = group_max_key<G>(best[0]);
          }
#pragma unroll
          for (int q = 0; q < V; ++q) key[q] = key[q] == best[0] ? 0 : key[q];
          slot[h] = l == j ? best[0] : slot[h];
        }
      }
    }
    float e[kHeld], taken = 0.0f;
    // a group of more lanes than sorted slots holds each slot once
    const bool holds = !kSort || l < kSorted;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      const bool some = holds && l + h * G < p.top_k && K::order_of(slot[h]) > K::kLow;
      e[h] = some ? exp_of(K::value(slot[h]) - top) : 0.0f;
      taken += e[h];
    }
    if (p.renorm) taken = group_sum<G>(taken);
    // a NaN among the logits is one of every weight
    const float f = p.renorm ? (total == total ? inverse(taken) : total) : inv;
    if (in) {
#pragma unroll
      for (int h = 0; h < kHeld; ++h) {
        const int32_t s = l + h * G;
        if (!holds || s >= p.top_k) continue;
        const bool some = counted && K::order_of(slot[h]) > K::kLow;
        const int32_t ex = some ? K::expert(slot[h]) : -1;
        p.idx[t * p.top_k + s] = ex;
        p.weights[t * p.top_k + s] = some ? e[h] * f : 0.0f;
        if (stats && some) atomicAdd(&counts[ex], 1);
      }
    }
  }
  if (!stats) return;
  // the wave's groups, then the block's waves, in a fixed order
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float s = sums[j];
    uint32_t a, b;
    if (G <= 8) {
      s += __shfl_xor(s, 8, 64);
    }
    if (G <= 16) {
      pair_of<16>(__float_as_uint(s), a, b);
      s = __uint_as_float(a) + __uint_as_float(b);
    }
    if (G <= 32) {
      pair_of<32>(__float_as_uint(s), a, b);
      s = __uint_as_float(a) + __uint_as_float(b);
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
    for (int w = 0; w < waves; ++w) s += prob[w][e];
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
struct RouteGradArgs {
  const void* logits;
  const int32_t* idx;
  const float* dweights;
  const int32_t* counts;
  const float* dloss;
  void* dlogits;
  uint32_t* status;
  int64_t ld, ld_d, n_tokens;
  int32_t n_experts, top_k;
  bool renorm, vec, vec_d;
};

// The slots' gradients reach their experts' lanes through a row of LDS a
// group: the sum of dweights of an expert's slots, and their number (a slot
// gets its gradient less the row's mean). The row is zero between tokens; its
// pieces of four are swizzled so that eight lanes' reads meet no bank twice.
// The next token's logits and slots are loaded while one is worked out.
// Measured: 65536 tokens of 256 bf16 experts, top 8, 27 us under the trace (71
// MB, 13.6 us of bytes; 494 vector instructions a wave's four rows, 14 us at
// the issue rate); 333 tokens of 60 fp32 experts 5.3.
template <int G, int V, bool kBf16, bool kOutBf16>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs p) {
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
  if (p.counts != nullptr) {
    const int32_t r = p.counts[p.n_experts];
    const float rows = static_cast<float>(r > 0 ? r : 1);
    const float f = p.dloss[0] * static_cast<float>(p.n_experts) /
                    (static_cast<float>(p.top_k) * rows) / rows;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (e0 + j < p.n_experts) load[j] = f * static_cast<float>(p.counts[e0 + j]);
  }
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
    float v[V], top = x.value(0);
#pragma unroll
    for (int j = 1; j < V; ++j) top = fmaxf(top, x.value(j));
    top = group_max<G>(top);
    float total = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v[j] = exp_of(x.value(j) - top);
      total += v[j];
    }
    const float inv = inverse(group_sum<G>(total));
    float u[V], hits[V], chosen = 0.0f, mean = 0.0f;
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      __builtin_memcpy(&u[4 * q], &grad_row[place(e0 + 4 * q)], 16);
      __builtin_memcpy(&hits[4 * q], &hits_row[place(e0 + 4 * q)], 16);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v[j] *= inv;
      chosen = __builtin_fmaf(hits[j], v[j], chosen);
      mean = __builtin_fmaf(u[j], v[j], mean);
    }
    if (p.renorm) {
      const float f = inverse(group_sum<G>(chosen));
      mean = group_sum<G>(mean) * f;
#pragma unroll
      for (int j = 0; j < V; ++j) u[j] = hits[j] != 0.0f ? (u[j] - hits[j] * mean) * f : 0.0f;
    }
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      u[j] += load[j];
      dot = __builtin_fmaf(v[j], u[j], dot);
    }
    dot = group_sum<G>(dot);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = counted ? v[j] * (u[j] - dot) : 0.0f;
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
          uint32_t d[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = pack_bf16(v[8 * b + 2 * j], v[8 * b + 2 * j + 1]);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dlogits) + row + ex) =
              uint4{d[0], d[1], d[2], d[3]};
        } else {
          __builtin_memcpy(__builtin_assume_aligned(static_cast<float*>(p.dlogits) + row + ex, 16),
                           &v[8 * b], 32);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (ex + j >= p.n_experts) continue;
          if (kOutBf16)
            static_cast<uint16_t*>(p.dlogits)[row + ex + j] = to_bf16_rne(v[8 * b + j]);
          else
            static_cast<float*>(p.dlogits)[row + ex + j] = v[8 * b + j];
        }
      }
    }
  }
}

// ------------------------------------------------------------------- hosts
// Lanes a row of the choice.
int32_t lanes_of(int32_t n_experts, bool bf16) {
  if (n_experts <= 64) return 8;
  const int32_t lanes = n_experts <= 128 ? 8 : n_experts <= 256 ? 16 : n_experts <= 512 ? 32 : 64;
  return bf16 || lanes == 64 ? lanes : 2 * lanes;
}

struct RouteShape {
  uint32_t blocks, threads;
};

RouteShape route_shape(int64_t n_tokens, int32_t n_experts, bool bf16) {
  const int64_t rows = 64 / lanes_of(n_experts, bf16), waves = (n_tokens + rows - 1) / rows;
  // up to four waves a block while that leaves a block for every CU
  const int64_t per = waves <= 1 ? 1 : waves <= 4 * kBlocks ? 4 : 16;
  int64_t blocks = (waves + per - 1) / per;
  if (blocks > kBlocks) blocks = kBlocks;
  return {static_cast<uint32_t>(blocks < 1 ? 1 : blocks), static_cast<uint32_t>(64 * per)};
}

template <int G, int V, typename K>
void launch_route(const RouteArgs& p, RouteShape s, hipStream_t st) {
  if (p.top_k <= kSorted)
    hipLaunchKernelGGL((route_kernel<G, V, K, true>), dim3(s.blocks), dim3(s.threads), 0, st, p);
  else
    hipLaunchKernelGGL((route_kernel<G, V, K, false>), dim3(s.blocks), dim3(s.threads), 0, st, p);
}

void launch_route_experts(const RouteArgs& p, RouteShape s, bool bf16, hipStream_t st) {
  const int32_t lanes = lanes_of(p.n_experts, bf16);
  if (bf16) {
    if (p.n_experts <= 64) launch_route<8, 8, KeyBf16>(p, s, st);
    else if (lanes == 8) launch_route<8, 16, KeyBf16>(p, s, st);
    else if (lanes == 16) launch_route<16, 16, KeyBf16>(p, s, st);
    else if (lanes == 32) launch_route<32, 16, KeyBf16>(p, s, st);
    else launch_route<64, 16, KeyBf16>(p, s, st);
  } else {
    if (p.n_experts <= 64) launch_route<8, 8, KeyF32>(p, s, st);
    else if (lanes == 16) launch_route<16, 8, KeyF32>(p, s, st);
    else if (lanes == 32) launch_route<32, 8, KeyF32>(p, s, st);
    else if (p.n_experts <= 512) launch_route<64, 8, KeyF32>(p, s, st);
    else launch_route<64, 16, KeyF32>(p, s, st);
  }
}

template <int G, int V>
void launch_grad(const RouteGradArgs& p, bool bf16, bool out_bf16, hipStream_t st) {
  // as many blocks as the chip holds: a wave's start (its experts' loads) is
  // worth several tokens (65536 x 256: 24 us; with 4096 blocks 42)
  const int64_t rows = 4 * (64 / G), b = (p.n_tokens + rows - 1) / rows;
  const dim3 grid(static_cast<uint32_t>(b < 1024 ? b : 1024)), block(256);
  if (bf16 && out_bf16) hipLaunchKernelGGL((route_grad_kernel<G, V, true, true>), grid, block, 0, st, p);
  else if (bf16) hipLaunchKernelGGL((route_grad_kernel<G, V, true, false>), grid, block, 0, st, p);
  else if (out_bf16) hipLaunchKernelGGL((route_grad_kernel<G, V, false, true>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((route_grad_kernel<G, V, false, false>), grid, block, 0, st, p);
}

}  // namespace
}  // namespace binade

using namespace binade;

extern "C" int64_t binade_moe_route_workspace_bytes(int64_t n_tokens, int32_t n_experts) {
  if (!route_sizes_ok(n_tokens, n_experts)) return 0;
  // Either type's call may have more blocks: fp32 rows take more lanes and with
  // them more waves, but above 1024 waves a block holds sixteen instead of four
  // (8192 tokens of 128 experts: 256 blocks in bf16, 128 in fp32).
  const int64_t f32 = route_shape(n_tokens, n_experts, false).blocks,
                bf16 = route_shape(n_tokens, n_experts, true).blocks;
  return kHead + (f32 > bf16 ? f32 : bf16) * (2 * n_experts + 1) * 4;
}

extern "C" int32_t binade_moe_route(const void* logits, int32_t dtype, int64_t ld, int64_t n_tokens,
                                    int32_t n_experts, int32_t top_k, int32_t renormalize,
                                    const uint8_t* valid, int32_t* idx, float* weights,
                                    int32_t* counts, float* prob_sum, float* loss, void* workspace,
                                    int64_t workspace_bytes, void* stream) {
  if (!route_sizes_ok(n_tokens, n_experts) || top_k < 1 || top_k > n_experts || top_k > kMaxTopK ||
      ld < n_experts)
    return BINADE_EINVAL;
  if (dtype != BINADE_F32 && dtype != BINADE_BF16) return BINADE_EINVAL;
  const bool stats = counts != nullptr;
  if (stats != (prob_sum != nullptr) || stats != (loss != nullptr)) return BINADE_EINVAL;
  if (n_tokens == 0 && !stats) return BINADE_OK;
  if (n_tokens > 0 && (logits == nullptr || idx == nullptr || weights == nullptr))
    return BINADE_EINVAL;
  if (stats) {
    if (workspace == nullptr ||
        workspace_bytes < binade_moe_route_workspace_bytes(n_tokens, n_experts))
      return BINADE_ENOSPACE;
    if (!aligned16(workspace)) return BINADE_EUNSUPPORTED;
  }
  const RouteShape shape = route_shape(n_tokens, n_experts, dtype == BINADE_BF16);
  RouteArgs p{};
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
  p.part_prob = reinterpret_cast<float*>(p.part_counts + static_cast<int64_t>(shape.blocks) *
                                                             (n_experts + 1));
  p.ld = ld;
  p.n_tokens = n_tokens;
  p.n_experts = n_experts;
  p.top_k = top_k;
  p.renorm = renormalize != 0;
  p.vec = whole_pieces(logits, n_experts, ld, dtype == BINADE_BF16);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  launch_route_experts(p, shape, dtype == BINADE_BF16, st);
  if (stats && shape.blocks > 1) {
    hipLaunchKernelGGL(route_stats_kernel, dim3(static_cast<uint32_t>((n_experts + 63) / 64)),
                       dim3(1024), 0, st, p, static_cast<int32_t>(shape.blocks));
  }
  return launch_status();
}

extern "C" int32_t binade_moe_route_grad(const void* logits, int32_t dtype, int64_t ld,
                                         int64_t n_tokens, int32_t n_experts, int32_t top_k,
                                         int32_t renormalize, const int32_t* idx,
                                         const float* dweights, const int32_t* counts,
                                         const float* dloss, void* dlogits, int32_t dlogits_dtype,
                                         int64_t ld_d, uint32_t* dev_status, void* stream) {
  if (!route_sizes_ok(n_tokens, n_experts) || top_k < 1 || top_k > n_experts || top_k > kMaxTopK ||
      ld < n_experts || ld_d < n_experts)
    return BINADE_EINVAL;
  if ((dtype != BINADE_F32 && dtype != BINADE_BF16) ||
      (dlogits_dtype != BINADE_F32 && dlogits_dtype != BINADE_BF16))
    return BINADE_EINVAL;
  if ((counts != nullptr) != (dloss != nullptr)) return BINADE_EINVAL;
  if (n_tokens == 0) return BINADE_OK;
  if (logits == nullptr || idx == nullptr || dlogits == nullptr) return BINADE_EINVAL;
  const bool bf16 = dtype == BINADE_BF16, out_bf16 = dlogits_dtype == BINADE_BF16;
  RouteGradArgs p{};
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
  p.renorm = renormalize != 0;
  p.vec = whole_pieces(logits, n_experts, ld, bf16);
  p.vec_d = whole_pieces(dlogits, n_experts, ld_d, out_bf16);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (n_experts <= 64) launch_grad<8, 8>(p, bf16, out_bf16, st);
  else if (n_experts <= 128) launch_grad<8, 16>(p, bf16, out_bf16, st);
  else if (n_experts <= 256) launch_grad<16, 16>(p, bf16, out_bf16, st);
  else if (n_experts <= 512) launch_grad<32, 16>(p, bf16, out_bf16, st);
  else launch_grad<64, 16>(p, bf16, out_bf16, st);
  return launch_status();
}
