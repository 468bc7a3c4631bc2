// Operators on the cache's FP8 rows: rotary positions with several axes, row packing and
// the join of partial attention results (the attention itself: ula_attend.cu).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cmath>
#include <utility>

#include "ula.h"

namespace {

constexpr uint32_t kPairs = ULA_ROPE_PAIRS;

// A rotary as the kernels take it: each pair's turns per position in 64-bit fixed point
// (2^64 = one turn), from a quotient in double.  position * step modulo 2^64 is then the angle's
// fraction of a turn in integer arithmetic: off by position * frequency * 1.5e-16 rad, the
// quotient's roundings (an fp32 product of position and frequency is off by up to 0.004 rad at
// position 10^5).
struct RotaryDev {
  unsigned long long step[kPairs];
  uint8_t axis[kPairs];
};

bool rotary_to_dev(const ula_rotary *r, RotaryDev *out) {
  if (!r || r->n_axes < 1 || r->n_axes > ULA_MAX_AXES || r->pairing > ULA_PAIR_HALVES) return false;
  for (uint32_t j = 0; j < kPairs; ++j) {
    if (r->axis[j] >= r->n_axes || !std::isfinite(r->freq[j])) return false;
    double turns = std::fabs((double)r->freq[j]) / 6.283185307179586476925286766559;
    turns -= std::floor(turns);
    const unsigned long long s =
        turns < 1.0 ? (unsigned long long)(turns * 18446744073709551616.0) : 0ull;
    out->step[j] = r->freq[j] < 0 ? 0ull - s : s;
    out->axis[j] = r->axis[j];
  }
  return true;
}

// (cos, sin) of a pair (of its step) at a position; the top 32 bits of the phase are the signed
// fraction of a turn, sincospi takes half turns in fp32 (24 bits: off by up to 9.4e-8 rad near half
// a turn, less for smaller angles).
__device__ __forceinline__ float2 turn_of(unsigned long long step, int32_t pos) {
  const unsigned long long phase = (unsigned long long)(long long)pos * step;
  const float half_turns = (float)(int32_t)(phase >> 32) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c, s);
}

// A pair turned.  Written out, so that the same operations are rounded in every kernel: left to the
// compiler, which product is fused differed from one to the other.
__device__ __forceinline__ void turn(float a, float b, float c, float s, float &oa, float &ob) {
  oa = fmaf(-b, s, __fmul_rn(a, c));
  ob = fmaf(b, c, __fmul_rn(a, s));
}

// Every kernel here may be launched while the one before it on the stream ends, and lets the
// next one do so: it waits before it touches memory.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f(float v) { return v; }

// ---------------------------------------------------------------- rotate

struct RotateParams {
  RotaryDev rot;
  const int32_t *pos;
  uint64_t pos_axis_stride;
  uint32_t n, heads;
  const void *x;
  uint64_t xt, xh;
  void *out;
  uint64_t ot, oh;
  float sign;  // -1 for the inverse
};

// 16 bytes of T, in fp32 and back.
template <typename T>
struct Vec {
  static constexpr int n = 16 / (int)sizeof(T);
  __device__ static __forceinline__ void open(const uint4 &u, float (&v)[n]) {
    const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = to_f(e[i]);
  }
  __device__ static __forceinline__ uint4 close(const float (&v)[n]) {
    uint4 u;
    T *e = reinterpret_cast<T *>(&u);
#pragma unroll
    for (int i = 0; i < n; ++i) e[i] = from_f<T>(v[i]);
    return u;
  }
};

// Bound by its bytes: every channel is read and written once.  A block takes `rows`
// consecutive (token, head) rows; its threads first issue their loads (kItems rows each,
// two 16-byte chunks of a row: channels of the first and of the second half), then work
// out the sines of the block's tokens together (once for all heads of a token), then turn
// and store.
template <typename T, bool kHalves, int kItems>
__global__ void __launch_bounds__(256) k_rotate_vec(const __grid_constant__ RotateParams p) {
  constexpr int V = Vec<T>::n, kPer = 32 / V;          // threads per row
  constexpr uint32_t kStep = 256 / kPer, kRows = kStep * kItems;
  extern __shared__ float4 table4[];                   // [tokens of the block][32] (cos, sin)
  float2 *table = reinterpret_cast<float2 *>(table4);
  const uint64_t all = (uint64_t)p.n * p.heads, row0 = (uint64_t)blockIdx.x * kRows;
  const uint64_t last = row0 + kRows < all ? row0 + kRows - 1 : all - 1;
  const uint32_t t0 = (uint32_t)(row0 / p.heads), t1 = (uint32_t)(last / p.heads);
  const uint32_t h0 = (uint32_t)(row0 - (uint64_t)t0 * p.heads);
  const uint32_t c = threadIdx.x % kPer, r0 = threadIdx.x / kPer;
  after_previous();
  uint4 lo[kItems], hi[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const uint32_t r = h0 + r0 + i * kStep, tok = r / p.heads;
    if (row0 + r0 + i * kStep < all) {
      const T *x = (const T *)p.x + (t0 + tok) * p.xt + (r - tok * p.heads) * p.xh + c * V;
      lo[i] = *reinterpret_cast<const uint4 *>(x);
      hi[i] = *reinterpret_cast<const uint4 *>(x + kPairs);
    }
  }
  // (a thread's pair is the same in every turn: the parameters' lane-wise reads, which the
  // constant port serves one lane at a time, are made once)
  const int32_t *pos = p.pos + p.rot.axis[threadIdx.x & 31] * p.pos_axis_stride + t0;
  const unsigned long long step = p.rot.step[threadIdx.x & 31];
  for (uint32_t k = threadIdx.x; k < (t1 - t0 + 1) * kPairs; k += 256) {
    float2 cs = turn_of(step, pos[k >> 5]);
    cs.y *= p.sign;
    table[k] = cs;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if (row0 + r0 + i * kStep >= all) break;
    const uint32_t r = h0 + r0 + i * kStep, tok = r / p.heads;
    const float4 *tb = table4 + tok * (kPairs / 2);
    float a[V], b[V], oa[V], ob[V];
    Vec<T>::open(lo[i], a);
    Vec<T>::open(hi[i], b);
    if (kHalves) {  // pair j: channel j of the first half with channel j of the second
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        const float4 cs = tb[(c * V + k) / 2];
        turn(a[k], b[k], cs.x, cs.y, oa[k], ob[k]);
        turn(a[k + 1], b[k + 1], cs.z, cs.w, oa[k + 1], ob[k + 1]);
      }
    } else {  // pair j: channels 2j, 2j + 1
      auto turn_pairs = [&](const float (&v)[V], float (&o)[V], uint32_t pair0) {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
          const float4 cs = tb[(pair0 + k / 2) / 2];
          turn(v[k], v[k + 1], cs.x, cs.y, o[k], o[k + 1]);
          turn(v[k + 2], v[k + 3], cs.z, cs.w, o[k + 2], o[k + 3]);
        }
      };
      turn_pairs(a, oa, c * (V / 2));
      turn_pairs(b, ob, kPairs / 2 + c * (V / 2));
    }
    T *o = (T *)p.out + (t0 + tok) * p.ot + (r - tok * p.heads) * p.oh + c * V;
    *reinterpret_cast<uint4 *>(o) = Vec<T>::close(oa);
    *reinterpret_cast<uint4 *>(o + kPairs) = Vec<T>::close(ob);
  }
}

// Any alignment and strides: one warp per token and head, one pair per lane.
template <typename T, bool kHalves>
__global__ void __launch_bounds__(256) k_rotate_any(const __grid_constant__ RotateParams p) {
  const uint64_t w = (uint64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const uint32_t j = threadIdx.x & 31;
  after_previous();
  if (w >= (uint64_t)p.n * p.heads) return;
  const uint32_t t = (uint32_t)(w / p.heads), h = (uint32_t)(w % p.heads);
  const T *x = (const T *)p.x + t * p.xt + h * p.xh;
  T *o = (T *)p.out + t * p.ot + h * p.oh;
  const float2 cs = turn_of(p.rot.step[j], p.pos[p.rot.axis[j] * p.pos_axis_stride + t]);
  const uint32_t ia = kHalves ? j : 2 * j, ib = kHalves ? j + kPairs : 2 * j + 1;
  float oa, ob;
  turn(to_f(x[ia]), to_f(x[ib]), cs.x, cs.y * p.sign, oa, ob);
  o[ia] = from_f<T>(oa);
  o[ib] = from_f<T>(ob);
}

// ---------------------------------------------------------------- pack

struct PackParams {
  RotaryDev rot;
  const int32_t *pos;
  uint64_t pos_axis_stride;
  uint32_t n;
  const void *latent;
  uint64_t latent_stride;
  const void *rope;
  uint64_t rope_stride;
  uint8_t *rows;
  uint64_t row_stride;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;  // (the second source goes to the low byte)
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Bound by its bytes.  One warp per token: lane l holds latents 16l..16l+15 (8 lanes share
// a block's scale) and turns rope pair l; a warp has the next token's loads in flight
// while it works on one.  kVec: 16-byte loads of the latents (bases and strides that allow
// them).  16 divisions a lane were half of the instructions; x / scale is the product with the
// scale's reciprocal and one correction by the remainder, which a fused multiply-add gives
// exactly (Markstein, IBM J. Res. Dev. 34, 1990): the correctly rounded quotient, so that a
// value near the middle of two codes goes to the nearer one.  (In blocks whose
// largest value is below about 2^-105 the remainder's last bits fall under the smallest number,
// and up to one quotient in 800 is off in its last bit.)
template <typename T, bool kHalves, bool kVec>
__global__ void __launch_bounds__(256) k_pack(const __grid_constant__ PackParams p) {
  constexpr int V = Vec<T>::n, N = 16 / V;
  const uint32_t l = threadIdx.x & 31, warps = gridDim.x * 8;
  const uint32_t ia = kHalves ? l : 2 * l, ib = kHalves ? l + kPairs : 2 * l + 1;
  uint4 next[N];
  T next_a, next_b;
  int32_t next_pos;
  const int32_t *posl = p.pos + p.rot.axis[l] * p.pos_axis_stride;
  const unsigned long long step = p.rot.step[l];
  auto fetch = [&](uint32_t t) {
    const T *x = (const T *)p.latent + t * p.latent_stride + 16 * l;
    const T *r = (const T *)p.rope + t * p.rope_stride;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (kVec) {
        next[i] = *reinterpret_cast<const uint4 *>(x + i * V);
      } else {
        T *e = reinterpret_cast<T *>(&next[i]);
#pragma unroll
        for (int k = 0; k < V; ++k) e[k] = x[i * V + k];
      }
    }
    next_a = r[ia], next_b = r[ib];
    next_pos = posl[t];
  };
  uint64_t t = (uint64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  after_previous();
  if (t < p.n) fetch((uint32_t)t);
  for (; t < p.n; t += warps) {
    float v[16], amax = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) Vec<T>::open(next[i], reinterpret_cast<float (&)[V]>(v[i * V]));
    const float a = to_f(next_a), b = to_f(next_b);
    const int32_t pos = next_pos;
    if (t + warps < p.n) fetch((uint32_t)(t + warps));
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = max_nan(amax, fabsf(v[i]));
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    const float scale = max_nan(__fdiv_rn(amax, 448.f), 0x1p-126f), inv = __frcp_rn(scale);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float q = v[i] * inv;
      v[i] = fmaf(fmaf(-q, scale, v[i]), inv, q);
    }
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    uint8_t *row = p.rows + t * p.row_stride;
    reinterpret_cast<uint4 *>(row)[l] = make_uint4(c[0], c[1], c[2], c[3]);
    if ((l & 7) == 0) reinterpret_cast<float *>(row + ULA_ROW_LATENT)[l >> 3] = scale;
    const float2 cs = turn_of(step, pos);
    __nv_bfloat16 *o = reinterpret_cast<__nv_bfloat16 *>(row + ULA_ROW_LATENT + 16);
    float oa, ob;
    turn(a, b, cs.x, cs.y, oa, ob);
    if (kHalves) {
      o[ia] = __float2bfloat16_rn(oa);
      o[ib] = __float2bfloat16_rn(ob);
    } else {
      reinterpret_cast<__nv_bfloat162 *>(o)[l] = __floats2bfloat162_rn(oa, ob);
    }
  }
}

// ---------------------------------------------------------------- join

struct JoinParams {
  const uint4 *outs[ULA_MAX_PARTS];
  const float *lses[ULA_MAX_PARTS];
  uint32_t parts;
  uint64_t n;
  uint4 *out;
  float *lse;
};

// 64 threads per query head, 8 channels each.
__global__ void __launch_bounds__(256) k_join(const __grid_constant__ JoinParams p) {
  const uint64_t i = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const uint32_t c = threadIdx.x & 63;
  after_previous();
  if (i >= p.n) return;
  uint4 v[ULA_MAX_PARTS];
  float z[ULA_MAX_PARTS], top = -INFINITY;
#pragma unroll
  for (uint32_t q = 0; q < ULA_MAX_PARTS; ++q)
    if (q < p.parts) {
      z[q] = p.lses[q][i];
      v[q] = p.outs[q][i * 64 + c];
    }
#pragma unroll
  for (uint32_t q = 0; q < ULA_MAX_PARTS; ++q)
    if (q < p.parts) top = max_nan(top, z[q]);
  const float ref = top == -INFINITY ? 0.f : top;
  float total = 0.f, acc[8] = {};
#pragma unroll
  for (uint32_t q = 0; q < ULA_MAX_PARTS; ++q)
    if (q < p.parts && z[q] != -INFINITY) {
      const float w = expf(z[q] - ref);
      total += w;
      const uint32_t u[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        acc[2 * k] += w * __uint_as_float(u[k] << 16);
        acc[2 * k + 1] += w * __uint_as_float(u[k] & 0xffff0000u);
      }
    }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  __nv_bfloat162 b[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) b[k] = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
  p.out[i * 64 + c] = *reinterpret_cast<uint4 *>(b);
  // (a part's lse may be the output: the row's 64 threads have all read theirs first)
  asm volatile("bar.sync %0, 64;" ::"r"(1 + (threadIdx.x >> 6)) : "memory");
  if (p.lse && c == 0) p.lse[i] = ref + logf(total);
}

template <typename P>
cudaError_t launch(void (*kernel)(P), uint64_t grid, uint32_t smem, cudaStream_t st, const P &p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

uint32_t type_size(uint32_t dtype) { return dtype == ULA_TYPE_F32 ? 4u : 2u; }
bool aligned(const void *p, uint64_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

uint32_t sm_count() {
  int dev = 0, n = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0
             ? (uint32_t)n : 1u;
}

// Whether two of the rows of 64 channels at i * si + j * sj (i < ni, j < nj) share elements.
bool overlap(uint64_t ni, uint64_t si, uint64_t nj, uint64_t sj) {
  constexpr uint64_t kRow = ULA_ROW_ROPE;
  if ((ni > 1 && si < kRow) || (nj > 1 && sj < kRow)) return true;
  if (ni < 2 || nj < 2) return false;
  if (si > sj) std::swap(si, sj), std::swap(ni, nj);
  using wide = unsigned __int128;
  if (sj >= (wide)(ni - 1) * si + kRow) return false;  // the rows of one j lie before those of the next
  const bool fewer_i = ni <= nj;                       // interleaved: every distance along the shorter side
  const uint64_t na = fewer_i ? ni : nj, nb = fewer_i ? nj : ni, sa = fewer_i ? si : sj, sb = fewer_i ? sj : si;
  for (uint64_t a = 1; a < na; ++a) {
    const wide at = (wide)a * sa, b = at / sb, below = at - b * sb;
    if ((b >= 1 && b < nb && below < kRow) || (b + 1 < nb && sb - below < kRow)) return true;
  }
  return false;
}

// Two rows per thread (4 loads in flight) where that leaves 4 blocks at least for every SM: 4,096
// tokens x 128 heads of bf16, 26.0 us (5.2 TB/s) against 29.3 with one and 27.8 with four.  Fewer
// rows are spread over more blocks of one row per thread, and so are tokens of few heads, whose
// sines would need more shared memory.
template <typename T, bool kHalves>
cudaError_t launch_rotate_vec(const RotateParams &p, cudaStream_t st) {
  const uint64_t all = (uint64_t)p.n * p.heads;
  constexpr uint32_t step = 256 / (32 / Vec<T>::n);
  const bool many = p.heads >= 8 && all >= 2ull * step * 4 * sm_count();
  const uint32_t rows = step * (many ? 2 : 1);
  const uint32_t tokens = (rows - 1) / p.heads + 2;  // at most, whatever the first row
  return launch(many ? k_rotate_vec<T, kHalves, 2> : k_rotate_vec<T, kHalves, 1>, (all + rows - 1) / rows,
                tokens * kPairs * 8, st, p);
}

template <typename T>
cudaError_t launch_rotate(const RotateParams &p, bool halves, bool vec, cudaStream_t st) {
  if (vec) return halves ? launch_rotate_vec<T, true>(p, st) : launch_rotate_vec<T, false>(p, st);
  const uint64_t blocks = ((uint64_t)p.n * p.heads + 7) / 8;
  return launch(halves ? k_rotate_any<T, true> : k_rotate_any<T, false>, blocks, 0, st, p);
}

template <typename T>
cudaError_t launch_pack(const PackParams &p, bool halves, bool vec, cudaStream_t st) {
  auto k = halves ? (vec ? k_pack<T, true, true> : k_pack<T, true, false>)
                  : (vec ? k_pack<T, false, true> : k_pack<T, false, false>);
  // a warp takes more than one token once every SM has its 4 resident blocks (131,072 tokens
  // of bf16: 42.6 us, 5.6 TB/s, with 4; 53.6 / 46.3 / 47.5 / 43.5 with 2 / 3 / 6 / 8)
  const uint64_t blocks = ((uint64_t)p.n + 7) / 8, most = 4ull * sm_count();
  return launch(k, blocks < most ? blocks : most, 0, st, p);
}

}  // namespace

extern "C" int ula_rows_rotate(const ula_rotary *rotary, uint32_t flags, const int32_t *d_pos,
                               uint64_t pos_axis_stride, uint32_t n, uint32_t heads,
                               uint32_t dtype, const void *d_x, uint64_t x_token_stride,
                               uint64_t x_head_stride, void *d_out, uint64_t out_token_stride,
                               uint64_t out_head_stride, void *stream) {
  RotateParams p{};
  if (!rotary_to_dev(rotary, &p.rot) || (flags & ~ULA_ROTATE_INVERSE) || dtype > ULA_TYPE_F32)
    return ULA_ERR_INVALID_ARG;
  const uint64_t work = (uint64_t)n * heads;
  if (work == 0) return ULA_OK;
  if (!d_pos || !d_x || !d_out || (work + 7) / 8 > 0x7fffffffull) return ULA_ERR_INVALID_ARG;
  if (!aligned(d_pos, 4) || !aligned(d_x, type_size(dtype)) || !aligned(d_out, type_size(dtype)))
    return ULA_ERR_INVALID_ARG;
  if (overlap(n, out_token_stride, heads, out_head_stride)) return ULA_ERR_INVALID_ARG;
  p.pos = d_pos, p.pos_axis_stride = pos_axis_stride, p.n = n, p.heads = heads;
  p.x = d_x, p.xt = x_token_stride, p.xh = x_head_stride;
  p.out = d_out, p.ot = out_token_stride, p.oh = out_head_stride;
  p.sign = (flags & ULA_ROTATE_INVERSE) ? -1.f : 1.f;
  const bool halves = rotary->pairing == ULA_PAIR_HALVES;
  const uint64_t strides = x_token_stride | x_head_stride | out_token_stride | out_head_stride;
  const bool vec = aligned(d_x, 16) && aligned(d_out, 16) && strides * type_size(dtype) % 16 == 0;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == ULA_TYPE_BF16  ? launch_rotate<__nv_bfloat16>(p, halves, vec, st)
                        : dtype == ULA_TYPE_F16 ? launch_rotate<__half>(p, halves, vec, st)
                                                : launch_rotate<float>(p, halves, vec, st);
  return e == cudaSuccess ? ULA_OK : ULA_ERR_CUDA;
}

extern "C" int ula_rows_pack(const ula_rotary *rotary, const int32_t *d_pos,
                             uint64_t pos_axis_stride, uint32_t n, uint32_t dtype,
                             const void *d_latent, uint64_t latent_stride, const void *d_rope,
                             uint64_t rope_stride, void *d_rows, uint64_t row_stride,
                             void *stream) {
  PackParams p{};
  if (!rotary_to_dev(rotary, &p.rot) || dtype > ULA_TYPE_F32) return ULA_ERR_INVALID_ARG;
  if (n == 0) return ULA_OK;
  if (!d_pos || !d_latent || !d_rope || !d_rows || row_stride < ULA_ROW_BYTES || row_stride % 16)
    return ULA_ERR_INVALID_ARG;
  if (!aligned(d_pos, 4) || !aligned(d_latent, type_size(dtype)) ||
      !aligned(d_rope, type_size(dtype)) || !aligned(d_rows, 16))
    return ULA_ERR_INVALID_ARG;
  p.pos = d_pos, p.pos_axis_stride = pos_axis_stride, p.n = n;
  p.latent = d_latent, p.latent_stride = latent_stride;
  p.rope = d_rope, p.rope_stride = rope_stride;
  p.rows = (uint8_t *)d_rows, p.row_stride = row_stride;
  const bool halves = rotary->pairing == ULA_PAIR_HALVES;
  const bool vec = aligned(d_latent, 16) && latent_stride * type_size(dtype) % 16 == 0;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == ULA_TYPE_BF16  ? launch_pack<__nv_bfloat16>(p, halves, vec, st)
                        : dtype == ULA_TYPE_F16 ? launch_pack<__half>(p, halves, vec, st)
                                                : launch_pack<float>(p, halves, vec, st);
  return e == cudaSuccess ? ULA_OK : ULA_ERR_CUDA;
}

extern "C" int ula_rows_join(const void *const *outs, const float *const *lses, uint32_t parts,
                             uint64_t n, void *out, float *lse, void *stream) {
  if (!outs || !lses || parts < 1 || parts > ULA_MAX_PARTS || (n + 3) / 4 > 0x7fffffffull)
    return ULA_ERR_INVALID_ARG;
  if (n == 0) return ULA_OK;
  JoinParams p{};
  for (uint32_t q = 0; q < parts; ++q) {
    if (!outs[q] || !lses[q] || !aligned(outs[q], 16) || !aligned(lses[q], 4)) return ULA_ERR_INVALID_ARG;
    p.outs[q] = (const uint4 *)outs[q];
    p.lses[q] = lses[q];
  }
  if (!out || !aligned(out, 16) || !aligned(lse, 4)) return ULA_ERR_INVALID_ARG;
  p.parts = parts, p.n = n, p.out = (uint4 *)out, p.lse = lse;
  return launch(k_join, (n + 3) / 4, 0, (cudaStream_t)stream, p) == cudaSuccess ? ULA_OK : ULA_ERR_CUDA;
}
