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
__global__ __launch_bounds__(256) void expand_kernel(LoraArgs p, const float* v, const uint16_t* w,
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
  return sizes_ok(m, n, k, rank) ? m * rank * 4 : 0;
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
  float* v = h != nullptr ? h : static_cast<float*>(workspace);
  hipLaunchKernelGGL(rows_kernel, dim3(static_cast<uint32_t>(m)), dim3(256), 0, st, p, x, ldx, p.a,
                     p.k, p.k, static_cast<int64_t>(1), false, v);
  hipLaunchKernelGGL(expand_kernel, dim3(blocks_for(m * p.n)), dim3(256), 0, st, p, v, p.b, p.n,
                     static_cast<int64_t>(1), static_cast<int64_t>(p.rank), true, base, ld_base,
                     base_dtype == BINADE_BF16, y, ldy, y_dtype == BINADE_BF16);
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
      hipLaunchKernelGGL(expand_kernel, dim3(blocks_for(m * p.k)), dim3(256), 0, st, p, g, p.a, p.k,
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
