// Accumulated attention weights (ula_rows_score): scores[address[e]] += sum over the query heads that
// select e of exp(z[e] - lse), with the logits z of ula_rows_attend and the lse that it gave.
//
// An address may be selected by several query tokens, so its weights are summed as 64-bit whole numbers
// (a fixed point that no sum of this call's weights can pass), whose sum does not depend on their
// order; one addition in fp32 per address then updates its score.  Three launches: the sums are cleared
// at the addresses in question, the weights are added, and each sum is taken by the first entry that
// finds it.
#include <cuda_bf16.h>
#include <cmath>

#include "ula.h"
#include "ula_tc.cuh"

using namespace ula_tc;

namespace {

struct ScoreParams {
  ula_score_args a;
  uint32_t lists, nodes;        // lists, and the query tokens of each
  unsigned long long *sums;     // [n_scores]
  float c0, unit;               // softmax_scale * log2(e); what 1.0 is in fixed point
};

__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__global__ void __launch_bounds__(256) k_score_clear(const __grid_constant__ ScoreParams p) {
  after_previous();
  const uint64_t n = (uint64_t)p.lists * p.a.k;
  for (uint64_t e = (uint64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (uint64_t)gridDim.x * 256) {
    const uint32_t a = (uint32_t)__ldg(p.a.address + e);
    if (a < p.a.n_scores) p.sums[a] = 0;
  }
}

// (Two calls that update the same scores at once: each adds its own sums.)
__global__ void __launch_bounds__(256) k_score_commit(const __grid_constant__ ScoreParams p) {
  after_previous();
  const uint64_t n = (uint64_t)p.lists * p.a.k;
  const double scale = 1.0 / (double)p.unit;
  for (uint64_t e = (uint64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (uint64_t)gridDim.x * 256) {
    const uint32_t a = (uint32_t)__ldg(p.a.address + e);
    if (a >= p.a.n_scores) continue;
    const unsigned long long s = atomicExch(p.sums + a, 0ull);
    if (s) atomicAdd(p.a.scores + a, (float)((double)s * scale));
  }
}

// A warp per entry: lane l holds latents 16l..16l+15 and two rope channels.
__global__ void __launch_bounds__(256) k_score(const __grid_constant__ ScoreParams p) {
  after_previous();
  const uint32_t lane = threadIdx.x & 31;
  const uint64_t n = (uint64_t)p.lists * p.a.k;
  const uint64_t e = (uint64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (e >= n) return;
  const uint32_t list = (uint32_t)(e / p.a.k);
  const uint32_t u = (uint32_t)__ldg(p.a.entry_row + e), to = (uint32_t)__ldg(p.a.address + e);
  if (u >= p.a.n_rows || to >= p.a.n_scores) return;
  const uint8_t *row = (const uint8_t *)p.a.rows + (uint64_t)u * ULA_ROW_BYTES;
  const uint4 codes = reinterpret_cast<const uint4 *>(row)[lane];
  const float scale = reinterpret_cast<const float *>(row + ULA_ROW_LATENT)[lane >> 3];
  const uint32_t rope = reinterpret_cast<const uint32_t *>(row + ULA_ROW_LATENT + 16)[lane];
  float v[18];
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t two = codes_to_bf16(w[i] >> (16 * h));
      v[4 * i + 2 * h] = __uint_as_float(two << 16), v[4 * i + 2 * h + 1] = __uint_as_float(two & 0xffff0000u);
    }
  v[16] = __uint_as_float(rope << 16), v[17] = __uint_as_float(rope & 0xffff0000u);
  const uint32_t req = list * p.nodes / p.a.n_q, first = list * p.nodes - req * p.a.n_q;
  float total = 0.f;
  for (uint32_t i = first; i < first + p.nodes; ++i)
    for (uint32_t h = 0; h < p.a.heads; ++h) {
      const __nv_bfloat16 *q = (const __nv_bfloat16 *)p.a.q + req * p.a.q_req_stride + i * p.a.q_tok_stride + h * p.a.q_head_stride;
      float x = 0.f;
#pragma unroll
      for (int c = 0; c < 16; ++c) x = fmaf(__bfloat162float(q[16 * lane + c]), v[c], x);
      x = x * scale + __bfloat162float(q[512 + 2 * lane]) * v[16] + __bfloat162float(q[513 + 2 * lane]) * v[17];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      const float lse = __ldg(p.a.lse + ((uint64_t)req * p.a.n_q + i) * p.a.heads + h);
      const float w1 = ex2(x * p.c0 - lse * 1.44269504088896341f);
      total += lse == -INFINITY || !(w1 > 0.f) ? 0.f : fminf(w1, 1.f);
    }
  if (lane == 0 && total > 0.f) atomicAdd(p.sums + to, __float2ull_rn(total * p.unit));
}

bool aligned(const void *p, uint64_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

cudaError_t launch(void (*kernel)(ScoreParams), uint64_t grid, cudaStream_t st, const ScoreParams &p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

extern "C" uint64_t ula_rows_score_workspace(uint32_t n_scores) { return (uint64_t)n_scores * 8; }

extern "C" int ula_rows_score(const ula_score_args *args, void *stream) {
  if (!args) return ULA_ERR_INVALID_ARG;
  ScoreParams p{};
  p.a = *args;
  ula_score_args &a = p.a;
  if (a.flags & ~ULA_TREE_SHARED_LIST) return ULA_ERR_INVALID_ARG;
  if (a.n_req == 1) a.q_req_stride = 0;  // (no steps: whatever they are)
  if (a.n_q == 1) a.q_tok_stride = 0;
  if (a.heads == 1) a.q_head_stride = 0;
  if (a.n_req == 0 || a.n_q == 0 || a.heads == 0 || a.k == 0 || a.n_scores == 0) return ULA_OK;
  if (!a.q || !a.entry_row || !a.address || !a.lse || !a.scores || !a.workspace || (!a.rows && a.n_rows))
    return ULA_ERR_INVALID_ARG;
  if (!aligned(a.q, 16) || !aligned(a.rows, 16) || !aligned(a.entry_row, 4) || !aligned(a.address, 4) ||
      !aligned(a.lse, 4) || !aligned(a.scores, 4) || !aligned(a.workspace, 8) || a.q_req_stride % 8 ||
      a.q_tok_stride % 8 || a.q_head_stride % 8 || a.n_rows > 0x7fffffffu || a.n_scores > 0x7fffffffu ||
      a.workspace_bytes < ula_rows_score_workspace(a.n_scores))
    return ULA_ERR_INVALID_ARG;
  const bool shared = a.flags & ULA_TREE_SHARED_LIST;
  const uint64_t tokens = (uint64_t)a.n_req * a.n_q;
  p.nodes = shared ? a.n_q : 1;
  if (tokens > 0x7fffffffull || a.heads > 0x7fffffffu || tokens * a.heads > 0x7fffffffull || a.k > 0x7fffffffu ||
      tokens * a.k > (1ull << 33))
    return ULA_ERR_INVALID_ARG;
  p.lists = shared ? a.n_req : (uint32_t)tokens;
  p.sums = (unsigned long long *)a.workspace;
  p.c0 = a.softmax_scale * 1.44269504088896341f;
  // a weight is at most 1, and an address gets at most one of every entry of every query head
  int bits = 0;
  while (bits < 62 && (double)tokens * a.heads * a.k > std::ldexp(1.0, bits)) ++bits;
  p.unit = std::ldexp(1.f, bits < 3 ? 60 : 63 - bits);
  const uint64_t n = (uint64_t)p.lists * a.k;
  cudaStream_t st = (cudaStream_t)stream;
  const uint64_t blocks = (n + 255) / 256 < 1024 ? (n + 255) / 256 : 1024;
  cudaError_t e = launch(k_score_clear, blocks, st, p);
  if (e == cudaSuccess) e = launch(k_score, (n + 7) / 8, st, p);
  if (e == cudaSuccess) e = launch(k_score_commit, blocks, st, p);
  return e == cudaSuccess ? ULA_OK : ULA_ERR_CUDA;
}
