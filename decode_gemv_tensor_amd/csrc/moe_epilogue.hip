// MoE epilogue: the gate.up activation between a MoE layer's expert
// products, and the top-k weighted combine after the down product.
//
// "Binade" package page (pypi.org/project/binade), "How it works" and
// "Limitations": a MoE layer's expert products (gate and up per chosen
// expert, then down) run as gathered matvecs; their outputs meet in an
// activation and, per token, in a sum over the chosen experts weighted by
// the router. Both steps are elementwise and HBM-bound; each thread owns
// outputs whose arithmetic is stated in binade.h:
//  - silu_mul: h = silu(g) * u with silu(g) = g / (1 + exp(-g)), in fp64 from
//    the fp32 inputs, rounded once to fp32 (then to bf16);
//  - combine: out[t, j] = fma chain over the token's top_k slots in slot
//    order from +0.0, in fp32 (then bf16).
// The combine's backward (what trains a router over these products) reads y
// and dout once and is HBM-bound too.
#include <hip/hip_runtime.h>

#include "binade.h"
#include "device_common.h"

namespace binade {
namespace {

using namespace dev;

__global__ __launch_bounds__(256) void silu_mul_kernel(const float* gate, const float* up,
                                                       int64_t n, void* h, int32_t h_bf16) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += stride) {
    const double g = gate[i];
    const double s = g / (1.0 + exp(-g));
    const float v = static_cast<float>(s * static_cast<double>(up[i]));
    if (h_bf16)
      static_cast<uint16_t*>(h)[i] = to_bf16_rne(v);
    else
      static_cast<float*>(h)[i] = v;
  }
}

__global__ __launch_bounds__(256) void combine_kernel(const float* y, const float* weights,
                                                      int64_t n_tokens, int32_t top_k, int64_t n,
                                                      void* out, int32_t out_bf16) {
  const int64_t total = n_tokens * n;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += stride) {
    const int64_t t = i / n, j = i - t * n;
    const float* wt = weights + t * top_k;
    const float* yt = y + t * top_k * n + j;
    float acc = 0.0f;
    for (int32_t s = 0; s < top_k; ++s) acc = __builtin_fmaf(wt[s], yt[s * n], acc);
    if (out_bf16)
      static_cast<uint16_t*>(out)[i] = to_bf16_rne(acc);
    else
      static_cast<float*>(out)[i] = acc;
  }
}

// dy[t, s, :] = w[t, s] * dout[t, :] and dw[t, s] = <dout[t, :], y[t, s, :]>:
// one block per (token, slot).
__global__ __launch_bounds__(256) void combine_grad_kernel(const float* y, const float* weights,
                                                           const void* dout, int32_t dout_bf16,
                                                           int32_t top_k, int64_t n, void* dy,
                                                           int32_t dy_bf16, float* dweights) {
  __shared__ float red[4];
  const int64_t pair = blockIdx.x, t = pair / top_k;
  const float w = weights[pair];
  float acc = 0.0f;
  for (int64_t j = threadIdx.x; j < n; j += 256) {
    const float d = dout_bf16 ? __uint_as_float(static_cast<uint32_t>(
                                    static_cast<const uint16_t*>(dout)[t * n + j]) << 16)
                              : static_cast<const float*>(dout)[t * n + j];
    acc = __builtin_fmaf(d, y[pair * n + j], acc);
    if (dy != nullptr) {
      if (dy_bf16)
        static_cast<uint16_t*>(dy)[pair * n + j] = to_bf16_rne(w * d);
      else
        static_cast<float*>(dy)[pair * n + j] = w * d;
    }
  }
  acc = slot_tree(acc);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
  __syncthreads();
  if (threadIdx.x == 0) dweights[pair] = ((red[0] + red[1]) + red[2]) + red[3];
}

uint32_t elementwise_blocks(int64_t n) {
  const int64_t b = (n + 255) / 256;
  return static_cast<uint32_t>(b < 8192 ? b : 8192);
}

}  // namespace
}  // namespace binade

using namespace binade;

extern "C" int32_t binade_moe_silu_mul(const float* gate, const float* up, int64_t n, void* h,
                                       int32_t h_dtype, void* stream) {
  if (n < 0 || (h_dtype != BINADE_F32 && h_dtype != BINADE_BF16)) return BINADE_EINVAL;
  if (n == 0) return BINADE_OK;
  if (gate == nullptr || up == nullptr || h == nullptr) return BINADE_EINVAL;
  hipLaunchKernelGGL(silu_mul_kernel, dim3(elementwise_blocks(n)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), gate, up, n, h,
                     static_cast<int32_t>(h_dtype == BINADE_BF16));
  return launch_status();
}

extern "C" int32_t binade_moe_combine(const float* y, const float* weights, int64_t n_tokens,
                                      int32_t top_k, int64_t n, void* out, int32_t out_dtype,
                                      void* stream) {
  if (n_tokens < 0 || n < 0 || top_k < 1 || top_k > 64) return BINADE_EINVAL;
  if (out_dtype != BINADE_F32 && out_dtype != BINADE_BF16) return BINADE_EINVAL;
  if (n_tokens == 0 || n == 0) return BINADE_OK;
  if (y == nullptr || weights == nullptr || out == nullptr) return BINADE_EINVAL;
  hipLaunchKernelGGL(combine_kernel, dim3(elementwise_blocks(n_tokens * n)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), y, weights, n_tokens, top_k, n, out,
                     static_cast<int32_t>(out_dtype == BINADE_BF16));
  return launch_status();
}

extern "C" int32_t binade_moe_combine_grad(const float* y, const float* weights, const void* dout,
                                           int32_t dout_dtype, int64_t n_tokens, int32_t top_k,
                                           int64_t n, void* dy, int32_t dy_dtype, float* dweights,
                                           void* stream) {
  if (n_tokens < 0 || n < 0 || top_k < 1 || top_k > 64) return BINADE_EINVAL;
  if ((dout_dtype != BINADE_F32 && dout_dtype != BINADE_BF16) ||
      (dy_dtype != BINADE_F32 && dy_dtype != BINADE_BF16))
    return BINADE_EINVAL;
  if (n_tokens * top_k > (1ll << 30) || n > (1ll << 30)) return BINADE_EUNSUPPORTED;
  if (n_tokens == 0) return BINADE_OK;
  if (dweights == nullptr || weights == nullptr) return BINADE_EINVAL;
  if (n > 0 && (y == nullptr || dout == nullptr)) return BINADE_EINVAL;
  hipLaunchKernelGGL(combine_grad_kernel, dim3(static_cast<uint32_t>(n_tokens * top_k)), dim3(256),
                     0, static_cast<hipStream_t>(stream), y, weights, dout,
                     static_cast<int32_t>(dout_dtype == BINADE_BF16), top_k, n, dy,
                     static_cast<int32_t>(dy_dtype == BINADE_BF16), dweights);
  return launch_status();
}
