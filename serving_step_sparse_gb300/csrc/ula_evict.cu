// Eviction by score (ula_rows_evict): which of a request's addresses stay.
//
// Of a list of n addresses, oldest first, the first `first` and the last `last` stay, and of the
// others those with the largest scores, `budget` in all; equal scores leave in order of place.  So the
// d = n - budget smallest (score, place) of the middle leave.  Scores become keys whose order as
// unsigned numbers is theirs; a radix select (11, 11 and 10 bits) finds the d-th smallest key T; then a
// stable partition by key < T, or key = T and fewer than the remaining ties before it, writes both
// lists.
//
// Bound by its bytes (12 an address: the address, its score, one of the outputs) and, for short lists,
// by the chain of a few passes.  A request's list is spread over a cluster of up to 8 blocks, so that
// 32 requests fill the GPU; keys are gathered once and stay in shared memory; histograms are summed
// through each other's shared memory.  The partition needs no barrier: a warp owns a run of places,
// knows how many of the runs before it leave, and goes on by ballots.
#include <cstdint>

#include <cuda_runtime.h>

#include "ula.h"

namespace {

constexpr uint32_t kThreads = 512, kWarps = kThreads / 32;
constexpr uint32_t kBins = 2048;                 // 4 a thread
constexpr uint32_t kMostCluster = 8;             // (the portable size)
constexpr uint32_t kMostKeys = 49152;            // a block's keys in shared memory, at most

struct EvictParams {
  const float *scores;
  uint32_t n_scores;
  const int32_t *address;       // [n_req][longest]
  const int32_t *length;        // [n_req]
  int32_t *kept, *dropped;      // [n_req][budget], [n_req][longest - budget]
  uint32_t longest, budget, first, last, dropped_room;
  bool cached;                  // the keys stand in shared memory
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t remote(uint32_t addr, uint32_t rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
  return at;
}
__device__ __forceinline__ uint32_t ld_remote(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_remote4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// A key per score, in the scores' order; -0 is 0, a NaN is larger than all numbers.
__device__ __forceinline__ uint32_t key_of(float s) {
  if (s != s) return 0xffffffffu;
  const uint32_t u = __float_as_uint(s + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Places of a warp's run, where `blocks` blocks share n: whole groups of 4 for every lane.
__host__ __device__ __forceinline__ uint32_t run_of(uint32_t n, uint32_t blocks) {
  return ((n + blocks * kWarps - 1) / (blocks * kWarps) + 127) & ~127u;
}

struct Smem {
  uint32_t hist[3][kBins];
  uint32_t warp[kWarps];        // a scan's sums
  uint32_t found[2];            // the digit, and how many keys below it
  uint32_t less[kWarps], equal[kWarps];
  uint32_t sums[2];             // the block's (less, equal)
};

template <bool kCluster>
__global__ void __launch_bounds__(kThreads) k_evict(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t raw[];
  Smem &s = *reinterpret_cast<Smem *>(raw);
  uint32_t *keys = raw + sizeof(Smem) / 4;
  uint32_t blocks = 1, rank = 0;
  if (kCluster) {
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(blocks));
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  }
  const uint32_t req = blockIdx.x / blocks;
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto meet = [] {
    __syncwarp();
    if (kCluster)
      asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
      __syncthreads();
  };
  for (uint32_t i = threadIdx.x; i < 3 * kBins; i += kThreads) (&s.hist[0][0])[i] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int32_t given = __ldg(p.length + req);
  const uint32_t n = given < 0 ? 0 : (uint32_t)given < p.longest ? (uint32_t)given : p.longest;
  const uint32_t leave = n > p.budget ? n - p.budget : 0;
  const int32_t *address = p.address + (uint64_t)req * p.longest;
  // a warp's run of places [run0, run1), the block's [begin, ...)
  const uint32_t run = run_of(n, blocks);
  const uint64_t block0 = (uint64_t)rank * kWarps * run, at0 = block0 + (uint64_t)warp * run;
  const uint32_t begin = block0 < n ? (uint32_t)block0 : n;
  const uint32_t run0 = at0 < n ? (uint32_t)at0 : n, run1 = at0 + run < n ? (uint32_t)at0 + run : n;
  const uint32_t mid0 = p.first, mid1 = n - (p.last < n ? p.last : n);  // places that may leave
  auto gather = [&](uint32_t i) -> uint32_t {
    const int32_t a = __ldg(address + i);
    return key_of((uint32_t)a < p.n_scores ? __ldg(p.scores + a) : 0.f);
  };
  auto key = [&](uint32_t i) -> uint32_t { return p.cached ? keys[i - begin] : gather(i); };
  auto four = [&](uint32_t i, uint32_t (&k)[4]) {  // places i.. (a multiple of 4) of the run
    if (p.cached) {
      *reinterpret_cast<uint4 *>(k) = *reinterpret_cast<const uint4 *>(keys + (i - begin));
    } else {
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) k[j] = i + j < run1 ? gather(i + j) : 0;
    }
  };
  auto middle = [&](uint32_t i) { return i >= mid0 && i < mid1; };

  uint32_t limit = 0, below = 0;  // T, and how many keys lie below it
  if (leave) {
    __syncthreads();  // (the histograms are clear)
    uint32_t digits = 0;
#pragma unroll
    for (uint32_t pass = 0; pass < 3; ++pass) {
      const uint32_t shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, mask = pass == 2 ? 1023 : 2047;
      auto count = [&](uint32_t k, bool in) {
        const uint32_t digit = (k >> shift) & mask;
        in = in && (pass == 0 || (k >> (pass == 1 ? 21 : 10)) == digits);
        // Most scores may be equal (addresses that were never selected), and adding to one place takes
        // a lane after the other: the digit of the first lane that has one is counted once for all of its lanes.
        uint32_t todo = __ballot_sync(0xffffffffu, in);
        if (todo) {
          const uint32_t lead = __ffs(todo) - 1, d = __shfl_sync(0xffffffffu, digit, lead);
          const uint32_t same = __ballot_sync(0xffffffffu, in && digit == d);
          if (lane == lead) atomicAdd(&s.hist[pass][d], __popc(same));
          if (in && digit != d) atomicAdd(&s.hist[pass][digit], 1u);
        }
      };
      if (pass == 0) {
        // eight gathers in flight, and the addresses of the next eight
        int32_t a[8];
        auto addresses = [&](uint32_t i0) {
#pragma unroll
          for (uint32_t j = 0; j < 8; ++j) {
            const uint32_t i = i0 + 32 * j + lane;
            a[j] = i < run1 ? __ldg(address + i) : -1;
          }
        };
        addresses(run0);
        for (uint32_t i0 = run0; i0 < run1; i0 += 256) {
          float v[8];
#pragma unroll
          for (uint32_t j = 0; j < 8; ++j) v[j] = (uint32_t)a[j] < p.n_scores ? __ldg(p.scores + a[j]) : 0.f;
          addresses(i0 + 256);
#pragma unroll
          for (uint32_t j = 0; j < 8; ++j) {
            const uint32_t i = i0 + 32 * j + lane, k = key_of(v[j]);
            if (p.cached && i < run1) keys[i - begin] = k;
            count(k, i < run1 && middle(i));
          }
        }
        __syncwarp();  // (a warp's keys are its own)
      } else {
        for (uint32_t i0 = run0; i0 < run1; i0 += 128) {
          uint32_t k[4];
          four(i0 + 4 * lane, k);
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t i = i0 + 4 * lane + j;
            count(k[j], i < run1 && middle(i));
          }
        }
      }
      meet();
      // the digit where the count of smaller keys passes what is still to leave
      uint4 c = make_uint4(0, 0, 0, 0);
      for (uint32_t r = 0; r < blocks; ++r) {
        const uint32_t at = smem_u32(&s.hist[pass][4 * threadIdx.x]);
        const uint4 v = kCluster ? ld_remote4(remote(at, r)) : *reinterpret_cast<const uint4 *>(&s.hist[pass][4 * threadIdx.x]);
        c.x += v.x, c.y += v.y, c.z += v.z, c.w += v.w;
      }
      const uint32_t mine = c.x + c.y + c.z + c.w;
      uint32_t sum = mine;
#pragma unroll
      for (uint32_t d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
      }
      if (lane == 31) s.warp[warp] = sum;
      __syncthreads();
      uint32_t before = sum - mine;
      for (uint32_t w = 0; w < warp; ++w) before += s.warp[w];
      const uint32_t want = leave - below;  // >= 1: the digit of the want-th smallest
      if (before < want && want <= before + mine) {
        uint32_t d = 4 * threadIdx.x;
        if (want > before + c.x) {
          before += c.x, ++d;
          if (want > before + c.y) {
            before += c.y, ++d;
            if (want > before + c.z) before += c.z, ++d;
          }
        }
        s.found[0] = d, s.found[1] = before;
      }
      __syncthreads();
      digits = (digits << (pass == 2 ? 10 : 11)) | s.found[0];
      below += s.found[1];
    }
    limit = digits;
  }

  // what leaves of the runs before this warp's
  uint32_t less = 0, equal = 0;
  if (leave) {
    for (uint32_t i0 = run0; i0 < run1; i0 += 128) {
      uint32_t k[4];
      four(i0 + 4 * lane, k);
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) {
        const uint32_t i = i0 + 4 * lane + j;
        const bool in = i < run1 && middle(i);
        less += in && k[j] < limit, equal += in && k[j] == limit;
      }
    }
    less = __reduce_add_sync(0xffffffffu, less), equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) s.less[warp] = less, s.equal[warp] = equal;
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t a = 0, b = 0;
      for (uint32_t w = 0; w < kWarps; ++w) a += s.less[w], b += s.equal[w];
      s.sums[0] = a, s.sums[1] = b;
    }
    meet();
    less = equal = 0;
    for (uint32_t r = 0; r < rank; ++r) {
      less += ld_remote(remote(smem_u32(&s.sums[0]), r));
      equal += ld_remote(remote(smem_u32(&s.sums[1]), r));
    }
    for (uint32_t w = 0; w < warp; ++w) less += s.less[w], equal += s.equal[w];
  }
  const uint32_t ties = leave - below;  // equal keys that leave: the first ones
  int32_t *kept = p.kept + (uint64_t)req * p.budget, *dropped = p.dropped + (uint64_t)req * p.dropped_room;
  const uint32_t before = (1u << lane) - 1;
  int32_t a[8];  // (the next addresses are on their way while these are placed)
  auto addresses = [&](uint32_t i0) {
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) {
      const uint32_t i = i0 + 32 * j + lane;
      a[j] = i < run1 ? __ldg(address + i) : -1;
    }
  };
  addresses(run0);
  for (uint32_t i0 = run0; i0 < run1; i0 += 256) {
    int32_t now[8];
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) now[j] = a[j];
    addresses(i0 + 256);
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) {
      const uint32_t i = i0 + 32 * j + lane;
      const bool in = leave && i < run1 && middle(i);
      const uint32_t k = in ? key(i) : 0;
      const uint32_t ls = __ballot_sync(0xffffffffu, in && k < limit), eq = __ballot_sync(0xffffffffu, in && k == limit);
      const uint32_t le = less + __popc(ls & before), ee = equal + __popc(eq & before);
      const bool goes = in && (k < limit || (k == limit && ee < ties));
      const uint32_t gone = le + (ee < ties ? ee : ties);  // before this place
      if (i < run1) (goes ? dropped + gone : kept + (i - gone))[0] = now[j];
      less += __popc(ls), equal += __popc(eq);
    }
  }
  for (uint32_t i = n - leave + rank * kThreads + threadIdx.x; i < p.budget; i += blocks * kThreads) kept[i] = -1;
  for (uint32_t i = leave + rank * kThreads + threadIdx.x; i < p.dropped_room; i += blocks * kThreads) dropped[i] = -1;
  if (kCluster) meet();  // (a block's shared memory stays until the others have read it)
}

bool aligned4(const void *p) { return ((uintptr_t)p & 3) == 0; }

}  // namespace

extern "C" int ula_rows_evict(const float *scores, uint32_t n_scores, const int32_t *address, const int32_t *length,
                              uint32_t n_req, uint32_t longest, uint32_t budget, uint32_t first, uint32_t last,
                              int32_t *kept, int32_t *dropped, void *stream) {
  if ((uint64_t)first + last > budget || longest > 0x7fffffffu || budget > 0x7fffffffu || n_scores > 0x7fffffffu)
    return ULA_ERR_INVALID_ARG;
  if (n_req == 0) return ULA_OK;
  EvictParams p{};
  p.scores = scores, p.n_scores = n_scores, p.address = address, p.length = length;
  p.kept = kept, p.dropped = dropped;
  p.longest = longest, p.budget = budget, p.first = first, p.last = last;
  p.dropped_room = longest > budget ? longest - budget : 0;
  if (!length || (n_scores && !scores) || (longest && !address) || (budget && !kept) || (p.dropped_room && !dropped) ||
      !aligned4(scores) || !aligned4(address) || !aligned4(length) || !aligned4(kept) || !aligned4(dropped))
    return ULA_ERR_INVALID_ARG;
  uint32_t cluster = 1;
  while (cluster < kMostCluster && longest > cluster * 2048) cluster *= 2;
  if ((uint64_t)n_req * cluster > 0x7fffffffull) return ULA_ERR_INVALID_ARG;
  const uint32_t run = run_of(longest, cluster);
  p.cached = (uint64_t)run * kWarps <= kMostKeys;
  const uint32_t smem = (uint32_t)sizeof(Smem) + (p.cached ? run * kWarps * 4 : 0);
  auto kernel = cluster > 1 ? k_evict<true> : k_evict<false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(sizeof(Smem) + kMostKeys * 4)) != cudaSuccess)
    return ULA_ERR_CUDA;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster, at[1].val.clusterDim.y = 1, at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(n_req * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? ULA_OK : ULA_ERR_CUDA;
}
