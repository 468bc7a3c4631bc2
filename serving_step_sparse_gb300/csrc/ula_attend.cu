// Attention over the cache's FP8 rows (ula_rows_attend).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ula.h"

namespace {

__device__ int g_status;  // the first error that a kernel of this file latched

constexpr uint32_t kChannels = ULA_ROW_LATENT + ULA_ROW_ROPE;

__device__ __forceinline__ float2 e4m3x2_to_f(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return __half22float2(*reinterpret_cast<__half2 *>(&h));
}

// One warp per query token and head: lane l holds latents 16l..16l+15 and rope channels
// 2l, 2l+1 of the query; one row at a time with a running maximum and sum.
__global__ void __launch_bounds__(256) k_attend(const ula_attend_args a) {
  const uint64_t w = (uint64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const uint32_t l = threadIdx.x & 31;
  const uint64_t n = (uint64_t)a.n_req * a.n_q * a.heads;
  if (w >= n) return;
  const uint32_t h = (uint32_t)(w % a.heads);
  const uint64_t tok = w / a.heads;
  const uint32_t r = (uint32_t)(tok / a.n_q), i = (uint32_t)(tok % a.n_q);
  const __nv_bfloat16 *q = (const __nv_bfloat16 *)a.q + r * a.q_req_stride + i * a.q_tok_stride + h * a.q_head_stride;
  float ql[16], acc[16] = {};
#pragma unroll
  for (int c = 0; c < 16; ++c) ql[c] = __bfloat162float(q[16 * l + c]);
  const float q0 = __bfloat162float(q[ULA_ROW_LATENT + 2 * l]), q1 = __bfloat162float(q[ULA_ROW_LATENT + 2 * l + 1]);
  float top = -INFINITY, total = 0.f;
  const uint32_t keys = a.k + (a.own_rows ? i + 1 : 0);
  for (uint32_t e = 0; e < keys; ++e) {
    const uint8_t *row;
    if (e < a.k) {
      const int32_t u = a.entry_row[tok * a.k + e];
      if (u < 0 || (uint32_t)u >= a.n_rows) continue;
      row = (const uint8_t *)a.rows + (uint64_t)u * ULA_ROW_BYTES;
    } else {
      row = (const uint8_t *)a.own_rows + r * a.own_req_stride + (e - a.k) * a.own_tok_stride;
    }
    const uint4 codes = reinterpret_cast<const uint4 *>(row)[l];
    const float s = reinterpret_cast<const float *>(row + ULA_ROW_LATENT)[l >> 3];
    const __nv_bfloat162 rope = reinterpret_cast<const __nv_bfloat162 *>(row + ULA_ROW_LATENT + 16)[l];
    const uint32_t cw[4] = {codes.x, codes.y, codes.z, codes.w};
    float v[16], z = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float2 lo = e4m3x2_to_f(cw[c] & 0xffffu), hi = e4m3x2_to_f(cw[c] >> 16);
      v[4 * c] = lo.x * s, v[4 * c + 1] = lo.y * s, v[4 * c + 2] = hi.x * s, v[4 * c + 3] = hi.y * s;
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) z += ql[c] * v[c];
    z += q0 * __low2float(rope) + q1 * __high2float(rope);
#pragma unroll
    for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
    z *= a.softmax_scale;
    const float up = fmaxf(top, z), ref = up == -INFINITY ? 0.f : up;
    const float f = expf(top - ref), p = expf(z - ref);
    top = up;
    total = total * f + p;
#pragma unroll
    for (int c = 0; c < 16; ++c) acc[c] = acc[c] * f + p * v[c];
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  __nv_bfloat162 o[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) o[c] = __floats2bfloat162_rn(acc[2 * c] * inv, acc[2 * c + 1] * inv);
  uint4 *out = reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.out + w * ULA_ROW_LATENT) + 2 * l;
  out[0] = reinterpret_cast<uint4 *>(o)[0];
  out[1] = reinterpret_cast<uint4 *>(o)[1];
  if (a.lse && l == 0) a.lse[w] = (top == -INFINITY ? 0.f : top) + logf(total);
}

bool aligned(const void *p, uint64_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace

extern "C" uint64_t ula_rows_attend_workspace(uint32_t n_req, uint32_t n_q, uint32_t heads,
                                              uint32_t k, int own) {
  (void)n_req, (void)n_q, (void)heads, (void)k, (void)own;
  return 0;
}

extern "C" int ula_rows_attend(const ula_attend_args *args, void *stream) {
  if (!args) return ULA_ERR_INVALID_ARG;
  const ula_attend_args &a = *args;
  const uint64_t tokens = (uint64_t)a.n_req * a.n_q;
  if (tokens == 0 || a.heads == 0) return ULA_OK;
  if (!a.q || !a.out || (a.k && (!a.entry_row || (!a.rows && a.n_rows)))) return ULA_ERR_INVALID_ARG;
  if (!aligned(a.q, 16) || !aligned(a.rows, 16) || !aligned(a.own_rows, 16) || !aligned(a.out, 16) ||
      !aligned(a.entry_row, 4) || !aligned(a.lse, 4) || !aligned(a.workspace, 16))
    return ULA_ERR_INVALID_ARG;
  if (a.q_req_stride % 8 || a.q_tok_stride % 8 || a.q_head_stride % 8 || a.own_req_stride % 16 ||
      a.own_tok_stride % 16 || a.n_rows > 0x7fffffffu || a.k > 0x7fffffffu - a.n_q)
    return ULA_ERR_INVALID_ARG;
  if (tokens > 0xffffffffull || (tokens * a.heads + 7) / 8 > 0x7fffffffull) return ULA_ERR_INVALID_ARG;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((tokens * a.heads + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = (cudaStream_t)stream;
  return cudaLaunchKernelEx(&cfg, k_attend, a) == cudaSuccess ? ULA_OK : ULA_ERR_CUDA;
}

extern "C" int ula_rows_sync(void *stream) {
  cudaStream_t st = (cudaStream_t)stream;
  int code = ULA_OK;
  const int none = ULA_OK;
  if (cudaMemcpyFromSymbolAsync(&code, g_status, sizeof code, 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return ULA_ERR_CUDA;
  if (code != ULA_OK &&
      (cudaMemcpyToSymbolAsync(g_status, &none, sizeof none, 0, cudaMemcpyHostToDevice, st) != cudaSuccess ||
       cudaStreamSynchronize(st) != cudaSuccess))
    return ULA_ERR_CUDA;
  return code;
}
