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

// Four values of a row from column j on (those below n) as fp32.
template <bool kBf16>
__device__ __forceinline__ void load4(const void* p, int64_t at, int64_t left, float (&f)[4]) {
  if (left >= 4) {
    if (kBf16) {
      uint32_t d[2];
      __builtin_memcpy(d, static_cast<const uint16_t*>(p) + at, 8);
      f[0] = bf16_lo(d[0]), f[1] = bf16_hi(d[0]), f[2] = bf16_lo(d[1]), f[3] = bf16_hi(d[1]);
    } else {
      __builtin_memcpy(f, static_cast<const float*>(p) + at, 16);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    f[j] = j >= left ? 0.0f
           : kBf16   ? __uint_as_float(
                         static_cast<uint32_t>(static_cast<const uint16_t*>(p)[at + j]) << 16)
                     : static_cast<const float*>(p)[at + j];
}

// Tokens along the grid's first axis, which ends at 2^32 threads.
constexpr int64_t kCombineRun = 1 << 17;

// dy[t, s, :] = w[t, s] * dout[t, :] and dw[t, s] = <dout[t, :], y[t, s, :]>:
// one block per token and S slots, which share the loads of dout; a thread
// has columns 4 threadIdx.x .. + 3 of every 1024. S does not change the order
// of a slot's sum. Blocks go to the 8 XCDs in turn, so a token's are 8 apart
// and find its dout in one L2 (1024 tokens of 8 slots 25.4 -> 23.2 us, 105 the
// same at 4096, as large as the caches above). Bound by y (read) and dy
// (written): 4096 tokens of 8 slots of 2816 columns, bf16 dout and dy, 105 us
// (577 MB, 5.5 TB/s).
template <int S, bool kDoutBf16, bool kDyBf16>
__global__ __launch_bounds__(256) void combine_grad_kernel(const float* y, const float* weights,
                                                           const void* dout, int64_t n_tokens,
                                                           int32_t top_k, int64_t n, void* dy,
                                                           float* dweights) {
  __shared__ float red[4][S];
  const int32_t chunks = (top_k + S - 1) / S;
  const uint32_t nth = blockIdx.x / 8;
  const int64_t t = blockIdx.y * kCombineRun + static_cast<int64_t>(nth / chunks) * 8 + blockIdx.x % 8;
  if (t >= n_tokens) return;
  const int32_t s0 = static_cast<int32_t>(nth % chunks) * S;
  const int32_t slots = top_k - s0 < S ? top_k - s0 : S;
  const int64_t pair = t * top_k + s0;
  float w[S], acc[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    w[s] = weights[pair + (s < slots ? s : 0)];
    acc[s] = 0.0f;
  }
  for (int64_t j = 4 * threadIdx.x; j < n; j += 1024) {
    float d[4], v[S][4];
    load4<kDoutBf16>(dout, t * n + j, n - j, d);
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (s < slots) load4<false>(y, (pair + s) * n + j, n - j, v[s]);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (s >= slots) break;
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[s] = __builtin_fmaf(d[q], v[s][q], acc[s]);
      if (dy == nullptr) continue;
      const int64_t at = (pair + s) * n + j;
      if (n - j >= 4) {
        if (kDyBf16) {
          uint32_t o[2];
#pragma unroll
          for (int q = 0; q < 2; ++q)
            o[q] = pack_bf16(w[s] * d[2 * q], w[s] * d[2 * q + 1]);
          __builtin_memcpy(static_cast<uint16_t*>(dy) + at, o, 8);
        } else {
          const float o[4] = {w[s] * d[0], w[s] * d[1], w[s] * d[2], w[s] * d[3]};
          __builtin_memcpy(static_cast<float*>(dy) + at, o, 16);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 3; ++q)
          if (j + q < n) {
            if (kDyBf16)
              static_cast<uint16_t*>(dy)[at + q] = to_bf16_rne(w[s] * d[q]);
            else
              static_cast<float*>(dy)[at + q] = w[s] * d[q];
          }
      }
    }
  }
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const float v = slot_tree(acc[s]);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][s] = v;
  }
  __syncthreads();
  if (static_cast<int32_t>(threadIdx.x) < slots) {
    const int s = threadIdx.x;
    dweights[pair + s] = ((red[0][s] + red[1][s]) + red[2][s]) + red[3][s];
  }
}

template <int S>
void launch_combine_grad(const float* y, const float* weights, const void* dout, bool dout_bf16,
                         int64_t n_tokens, int32_t top_k, int64_t n, void* dy, bool dy_bf16,
                         float* dweights, hipStream_t st) {
  const int64_t run = n_tokens < kCombineRun ? (n_tokens + 7) / 8 * 8 : kCombineRun;
  const dim3 grid(static_cast<uint32_t>(run * ((top_k + S - 1) / S)),
                  static_cast<uint32_t>((n_tokens + kCombineRun - 1) / kCombineRun)),
      block(256);
  if (dout_bf16 && dy_bf16)
    hipLaunchKernelGGL((combine_grad_kernel<S, true, true>), grid, block, 0, st, y, weights, dout,
                       n_tokens, top_k, n, dy, dweights);
  else if (dout_bf16)
    hipLaunchKernelGGL((combine_grad_kernel<S, true, false>), grid, block, 0, st, y, weights, dout,
                       n_tokens, top_k, n, dy, dweights);
  else if (dy_bf16)
    hipLaunchKernelGGL((combine_grad_kernel<S, false, true>), grid, block, 0, st, y, weights, dout,
                       n_tokens, top_k, n, dy, dweights);
  else
    hipLaunchKernelGGL((combine_grad_kernel<S, false, false>), grid, block, 0, st, y, weights, dout,
                       n_tokens, top_k, n, dy, dweights);
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
  if (n_tokens > (1ll << 30) / top_k || n > (1ll << 30)) return BINADE_EUNSUPPORTED;
  if (n_tokens == 0) return BINADE_OK;
  if (dweights == nullptr || weights == nullptr) return BINADE_EINVAL;
  if (n > 0 && (y == nullptr || dout == nullptr)) return BINADE_EINVAL;
  const bool db = dout_dtype == BINADE_BF16, yb = dy_dtype == BINADE_BF16;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  // a block per slot until the tokens alone fill the chip (8 slots of 2816
  // columns: 8 tokens 4.4 us, with eight a block 10.3; 256 tokens 8.2, with two
  // 8.9; 4096 tokens 109, with two 105, four 111, eight 121)
  if (n_tokens < 512)
    launch_combine_grad<1>(y, weights, dout, db, n_tokens, top_k, n, dy, yb, dweights, st);
  else
    launch_combine_grad<2>(y, weights, dout, db, n_tokens, top_k, n, dy, yb, dweights, st);
  return launch_status();
}
