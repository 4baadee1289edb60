// The router of a MoE layer and its backward: softmax, top-k, per-expert
// counts, balance loss (the arithmetic is stated in binade.h).
//
// One wave per row; a lane holds the row's experts lane, lane + 64, ...
// (at most 16 of 1024).
#include <hip/hip_runtime.h>

#include "binade.h"
#include "device_common.h"

namespace binade {
namespace {

using namespace dev;

constexpr int kMaxExperts = 1024;
constexpr int kPerLane = kMaxExperts / 64;
constexpr int kMaxTopK = 64;
constexpr int32_t kPartBlocks = 256;   // blocks that keep a row of partial sums each

struct RouteArgs {
  const void* logits;
  const uint8_t* valid;
  int32_t* idx;
  float* weights;
  int32_t* part_counts;   // [blocks, n_experts + 1] or NULL
  float* part_prob;       // [blocks, n_experts]
  int64_t ld, n_tokens;
  int32_t n_experts, top_k;
  bool bf16, renorm;
};

__device__ __forceinline__ float load_logit(const void* p, int64_t i, bool bf16) {
  return bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16)
              : static_cast<const float*>(p)[i];
}

// Ordered key of (logit, expert): larger logit first, then the smaller
// expert; 0 for an expert that cannot be taken (-inf or NaN).
__device__ __forceinline__ uint64_t key_of(float v, int32_t e) {
  if (!(v > -__builtin_inff())) return 0;
  v = v + 0.0f;   // -0 -> +0: equal logits tie
  const uint32_t u = __float_as_uint(v);
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return (static_cast<uint64_t>(o) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(e));
}

__device__ __forceinline__ uint64_t wave_max(uint64_t k) {
  for (int s = 32; s >= 1; s >>= 1) {
    const uint64_t o = __shfl_xor(static_cast<unsigned long long>(k), s, 64);
    k = o > k ? o : k;
  }
  return k;
}

__device__ __forceinline__ float wave_sum(float v) {
  for (int s = 32; s >= 1; s >>= 1) v = v + __shfl_xor(v, s, 64);
  return v;
}

__global__ __launch_bounds__(256) void route_kernel(RouteArgs p) {
  __shared__ int32_t counts[kMaxExperts + 1];
  __shared__ float prob[4][kMaxExperts];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int32_t e = threadIdx.x; e <= p.n_experts; e += 256) counts[e] = 0;
  __syncthreads();
  float sums[kPerLane];
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) sums[j] = 0.0f;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave; t < p.n_tokens;
       t += static_cast<int64_t>(gridDim.x) * 4) {
    const bool valid = p.valid == nullptr || p.valid[t] != 0;
    float v[kPerLane];
    uint64_t key[kPerLane];
    bool nan = false;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const int32_t e = lane + 64 * j;
      v[j] = e < p.n_experts ? load_logit(p.logits, t * p.ld + e, p.bf16) : -__builtin_inff();
      nan |= v[j] != v[j];
      key[j] = key_of(v[j], e);
    }
    uint64_t best = 0;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) best = key[j] > best ? key[j] : best;
    best = wave_max(best);
    const bool counted = valid && best != 0;
    int32_t* idx = p.idx + t * p.top_k;
    float* w = p.weights + t * p.top_k;
    if (!counted) {
      if (lane < p.top_k) idx[lane] = -1, w[lane] = 0.0f;
      continue;
    }
    const uint32_t o = static_cast<uint32_t>(best >> 32);
    const float top = __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
    float total = 0.0f, pr[kPerLane];
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      pr[j] = expf(v[j] - top);
      total += pr[j];
    }
    total = wave_sum(total);
    float mine = 0.0f, taken = 0.0f;   // lane s: the weight of slot s
    int32_t my_idx = -1;
    for (int32_t s = 0; s < p.top_k; ++s) {
      if (s > 0) {
        best = 0;
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) best = key[j] > best ? key[j] : best;
        best = wave_max(best);
      }
      if (best == 0) break;
      const int32_t e = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(best));
      float pe = 0.0f;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j)
        if (key[j] == best) key[j] = 0, pe = pr[j];
      pe = __shfl(pe, e & 63, 64) / total;
      taken += pe;
      if (lane == s) mine = pe, my_idx = e;
    }
    if (lane < p.top_k) {
      idx[lane] = my_idx;
      w[lane] = my_idx < 0 ? 0.0f : p.renorm ? mine / taken : mine;
    }
    if (p.part_counts != nullptr) {
      if (my_idx >= 0) atomicAdd(&counts[my_idx], 1);
      if (lane == 0) atomicAdd(&counts[p.n_experts], 1);
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) sums[j] += pr[j] / total;
    }
  }
  if (p.part_counts == nullptr) return;
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) prob[wave][lane + 64 * j] = sums[j];
  __syncthreads();
  for (int32_t e = threadIdx.x; e <= p.n_experts; e += 256) {
    p.part_counts[static_cast<int64_t>(blockIdx.x) * (p.n_experts + 1) + e] = counts[e];
    if (e < p.n_experts)
      p.part_prob[static_cast<int64_t>(blockIdx.x) * p.n_experts + e] =
          ((prob[0][e] + prob[1][e]) + prob[2][e]) + prob[3][e];
  }
}

// Adds the blocks' partial counts and sums in block order; the loss is a
// fixed tree over the experts. One block.
__global__ __launch_bounds__(1024) void route_stats_kernel(const int32_t* part_counts,
                                                           const float* part_prob, int32_t blocks,
                                                           int32_t n_experts, int32_t top_k,
                                                           int32_t* counts, float* prob_sum,
                                                           float* loss) {
  __shared__ float red[16];
  __shared__ int32_t rows_s;
  const int32_t e = threadIdx.x;
  if (e == 0) {
    int32_t rows = 0;
    for (int32_t b = 0; b < blocks; ++b)
      rows += part_counts[static_cast<int64_t>(b) * (n_experts + 1) + n_experts];
    rows_s = rows;
    counts[n_experts] = rows;
  }
  int32_t c = 0;
  float s = 0.0f;
  if (e < n_experts) {
    for (int32_t b = 0; b < blocks; ++b) {
      c += part_counts[static_cast<int64_t>(b) * (n_experts + 1) + e];
      s += part_prob[static_cast<int64_t>(b) * n_experts + e];
    }
    counts[e] = c;
    prob_sum[e] = s;
  }
  __syncthreads();
  const float rows = static_cast<float>(rows_s > 0 ? rows_s : 1);
  const float part = wave_sum(static_cast<float>(c) / (static_cast<float>(top_k) * rows) *
                              (s / rows));
  if ((e & 63) == 0) red[e >> 6] = part;
  __syncthreads();
  if (e == 0) {
    float l = 0.0f;
    for (int w = 0; w < 16; ++w) l += red[w];
    loss[0] = static_cast<float>(n_experts) * l;
  }
}

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
  bool bf16, d_bf16, renorm;
};

__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float load[kPerLane];
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) load[j] = 0.0f;
  if (p.counts != nullptr) {
    const int32_t r = p.counts[p.n_experts];
    const float rows = static_cast<float>(r > 0 ? r : 1);
    const float f = p.dloss[0] * static_cast<float>(p.n_experts) /
                    (static_cast<float>(p.top_k) * rows * rows);
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const int32_t e = lane + 64 * j;
      if (e < p.n_experts) load[j] = f * static_cast<float>(p.counts[e]);
    }
  }
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave; t < p.n_tokens;
       t += static_cast<int64_t>(gridDim.x) * 4) {
    int32_t e_s = -1;
    float dw = 0.0f;
    if (lane < p.top_k) {
      e_s = p.idx[t * p.top_k + lane];
      if (e_s >= p.n_experts || e_s < 0) {
        if (e_s != -1 && p.status != nullptr)
          atomicOr(p.status, static_cast<uint32_t>(BINADE_DEV_BAD_INDEX));
        e_s = -1;
      }
      if (p.dweights != nullptr) dw = p.dweights[t * p.top_k + lane];
    }
    const bool counted = __shfl(e_s, 0, 64) >= 0;
    float v[kPerLane];
    float top = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const int32_t e = lane + 64 * j;
      v[j] = e < p.n_experts ? load_logit(p.logits, t * p.ld + e, p.bf16) : -__builtin_inff();
      top = fmaxf(top, v[j]);
    }
    for (int s = 32; s >= 1; s >>= 1) top = fmaxf(top, __shfl_xor(top, s, 64));
    float total = 0.0f;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      v[j] = expf(v[j] - top);
      total += v[j];
    }
    total = wave_sum(total);
    float u[kPerLane];
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      v[j] = v[j] / total;
      u[j] = load[j];
    }
    float chosen = 0.0f;   // lane s: p of slot s
    if (p.renorm) {
      for (int32_t s = 0; s < p.top_k; ++s) {
        const int32_t e = __shfl(e_s, s, 64);
        if (e < 0) continue;
        float pe = 0.0f;
#pragma unroll
        for (int j = 0; j < kPerLane; ++j)
          if (e == lane + 64 * j) pe = v[j];
        pe = __shfl(pe, e & 63, 64);
        if (lane == s) chosen = pe;
      }
      const float sum = wave_sum(chosen);
      const float mean = wave_sum(e_s >= 0 ? dw * chosen / sum : 0.0f);
      dw = (dw - mean) / sum;
    }
    for (int32_t s = 0; s < p.top_k; ++s) {
      const int32_t e = __shfl(e_s, s, 64);
      const float d = __shfl(dw, s, 64);
      if (e < 0) continue;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j)
        if (e == lane + 64 * j) u[j] += d;
    }
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) dot = __builtin_fmaf(v[j], u[j], dot);
    dot = wave_sum(dot);
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const int32_t e = lane + 64 * j;
      if (e >= p.n_experts) continue;
      const float d = counted ? v[j] * (u[j] - dot) : 0.0f;
      if (p.d_bf16)
        static_cast<uint16_t*>(p.dlogits)[t * p.ld_d + e] = to_bf16_rne(d);
      else
        static_cast<float*>(p.dlogits)[t * p.ld_d + e] = d;
    }
  }
}

uint32_t route_blocks(int64_t n_tokens) {
  const int64_t b = (n_tokens + 3) / 4;
  return static_cast<uint32_t>(b < 1 ? 1 : b < kPartBlocks ? b : kPartBlocks);
}

bool route_sizes_ok(int64_t n_tokens, int32_t n_experts) {
  return n_tokens >= 0 && n_tokens <= (1ll << 30) && n_experts >= 1 && n_experts <= kMaxExperts;
}

}  // namespace
}  // namespace binade

using namespace binade;

extern "C" int64_t binade_moe_route_workspace_bytes(int64_t n_tokens, int32_t n_experts) {
  if (!route_sizes_ok(n_tokens, n_experts)) return 0;
  return static_cast<int64_t>(route_blocks(n_tokens)) * (2 * n_experts + 1) * 4;
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
  const uint32_t blocks = route_blocks(n_tokens);
  RouteArgs p{};
  p.logits = logits;
  p.valid = valid;
  p.idx = idx;
  p.weights = weights;
  if (stats) {
    p.part_counts = static_cast<int32_t*>(workspace);
    p.part_prob =
        reinterpret_cast<float*>(p.part_counts + static_cast<int64_t>(blocks) * (n_experts + 1));
  }
  p.ld = ld;
  p.n_tokens = n_tokens;
  p.n_experts = n_experts;
  p.top_k = top_k;
  p.bf16 = dtype == BINADE_BF16;
  p.renorm = renormalize != 0;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(route_kernel, dim3(blocks), dim3(256), 0, st, p);
  if (stats)
    hipLaunchKernelGGL(route_stats_kernel, dim3(1), dim3(1024), 0, st, p.part_counts, p.part_prob,
                       static_cast<int32_t>(blocks), n_experts, top_k, counts, prob_sum, loss);
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
  p.bf16 = dtype == BINADE_BF16;
  p.d_bf16 = dlogits_dtype == BINADE_BF16;
  p.renorm = renormalize != 0;
  const int64_t b = (n_tokens + 3) / 4;
  hipLaunchKernelGGL(route_grad_kernel, dim3(static_cast<uint32_t>(b < 2048 ? b : 2048)), dim3(256),
                     0, static_cast<hipStream_t>(stream), p);
  return launch_status();
}
