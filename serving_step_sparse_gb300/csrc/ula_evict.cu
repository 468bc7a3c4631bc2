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
// 32 requests fill the GPU; keys are gathered once and stay in shared memory; histograms are summed in
// the first block's (each block reading all of them took 5,000 to 13,000 clocks a pass).  The partition needs no barrier: a warp owns a run of places,
// knows how many of the runs before it leave, and goes on by ballots.  32 lists of 65,536 to 131,072 addresses,
// 39,321 of each kept: 29 us (0.2 of the copy rate): the longest list's gathers, three passes with two
// meetings each, and the partition follow each other (17,000, 18,000 and 10,000 clocks).
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
__device__ __forceinline__ void add_remote(uint32_t at, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void st_remote2(uint32_t at, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(a), "r"(b) : "memory");
}

// A key per score, in the scores' order; -0 is 0, a NaN is larger than all numbers.  kStays is larger than
// every key: a place that may not leave, or lies behind the list.
constexpr uint32_t kStays = 0xffffffffu, kZero = 0x80000000u;
__device__ __forceinline__ uint32_t key_of(float s) {
  const uint32_t u = __float_as_uint(s + 0.f);
  const uint32_t k = u ^ (uint32_t)((int32_t)u >> 31 | (int32_t)0x80000000);
  return s == s ? k : kStays - 1;
}

// Places of a warp's run, where `blocks` blocks share n: whole groups of 4 for every lane.
__host__ __device__ __forceinline__ uint32_t run_of(uint32_t n, uint32_t blocks) {
  return ((n + blocks * kWarps - 1) / (blocks * kWarps) + 127) & ~127u;
}

struct Smem {
  uint32_t hist[2][kBins];      // a pass's of this block; in the first block, their sum
  uint32_t warp[kWarps];        // a scan's sums
  uint2 found[3];               // a pass's digit, and how many keys below it
  uint2 sums[kWarps][kMostCluster];  // the runs' (less, equal)
  uint2 pad;                    // (the keys start on 16 bytes)
};
static_assert(sizeof(Smem) % 16 == 0, "keys are read by fours");

template <bool kCluster>
__global__ void __launch_bounds__(kThreads) k_evict(const __grid_constant__ EvictParams p) {
  extern __shared__ uint4 raw[];
  Smem &s = *reinterpret_cast<Smem *>(raw);
  uint32_t *keys = reinterpret_cast<uint32_t *>(raw) + sizeof(Smem) / 4;
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
  for (uint32_t i = threadIdx.x; i < 2 * kBins; i += kThreads) (&s.hist[0][0])[i] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int32_t given = __ldg(p.length + req);
  const uint32_t n = given < 0 ? 0 : (uint32_t)given < p.longest ? (uint32_t)given : p.longest;
  const uint32_t leave = n > p.budget ? n - p.budget : 0;
  const int32_t *address = p.address + (uint64_t)req * p.longest;
  // A warp's run of places [run0, run1), and where its keys stand.  The blocks take the runs in turn: a
  // list's last places were written one at a time, with other requests' between them, and their scores
  // take a load each where a prompt's share one.
  const uint32_t run = run_of(n, blocks);
  const uint64_t at0 = ((uint64_t)warp * blocks + rank) * run;
  const uint32_t run0 = at0 < n ? (uint32_t)at0 : n, run1 = at0 + run < n ? (uint32_t)at0 + run : n;
  uint32_t *const mine = keys + warp * run;
  const uint32_t mid0 = p.first, mid1 = n - (p.last < n ? p.last : n);  // places that may leave
  // addresses of the places i0 + lane, i0 + 32 + lane, ... (-1 behind the run); scores; the key of place i
  auto addresses = [&](uint32_t i0, auto &a) {
#pragma unroll
    for (uint32_t j = 0; j < sizeof a / 4; ++j) {
      const uint32_t i = i0 + 32 * j + lane;
      a[j] = i < run1 ? __ldg(address + i) : -1;
    }
  };
  auto score = [&](int32_t a) { return (uint32_t)a < p.n_scores ? __ldg(p.scores + a) : 0.f; };
  auto key_at = [&](uint32_t i, float v) { return i >= mid0 && i < mid1 && i < run1 ? key_of(v) : kStays; };
  auto four = [&](uint32_t i, uint32_t (&k)[4]) {  // the keys of places i..
    if (p.cached) {
      *reinterpret_cast<uint4 *>(k) = *reinterpret_cast<const uint4 *>(mine + (i - run0));
    } else {
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) k[j] = key_at(i + j, i + j < run1 ? score(__ldg(address + i + j)) : 0.f);
    }
  };

  uint32_t limit = 0, below = 0;  // T, and how many keys lie below it
  if (leave) {
    meet();  // (the histograms are clear)
    uint32_t digits = 0, zeros = 0;
#pragma unroll
    for (uint32_t pass = 0; pass < 3; ++pass) {
      const uint32_t shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, mask = pass == 2 ? 1023 : 2047;
      // Many scores may be equal (addresses that were never selected have 0), and adding to one place takes
      // a lane after the other: zeros are counted in a register.
      auto count = [&](uint32_t k) {
        if (pass == 0 && k == kZero) ++zeros;
        else if (pass == 0 || ((k >> (pass == 1 ? 21 : 10)) == digits && k != kZero)) atomicAdd(&s.hist[0][(k >> shift) & mask], 1u);
      };
      if (pass == 0) {
        // sixteen gathers in flight, and the addresses of the next sixteen
        int32_t a[16];
        addresses(run0, a);
        for (uint32_t i0 = run0; i0 < run1; i0 += 512) {
          float v[16];
#pragma unroll
          for (uint32_t j = 0; j < 16; ++j) v[j] = score(a[j]);
          addresses(i0 + 512, a);
#pragma unroll
          for (uint32_t j = 0; j < 16; ++j) {
            const uint32_t i = i0 + 32 * j + lane, k = key_at(i, v[j]);
            if (p.cached && i0 + (j & ~3u) * 32 < run1) mine[i - run0] = k;  // (a run is whole groups of 128 places)
            count(k);
          }
        }
        __syncwarp();  // (a warp's keys are its own)
        zeros = __reduce_add_sync(0xffffffffu, zeros);
      } else {
        for (uint32_t i0 = run0; i0 < run1; i0 += 128) {
          uint32_t k[4];
          four(i0 + 4 * lane, k);
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) count(k[j]);
        }
      }
      if (lane == 0 && zeros && (pass == 0 || (kZero >> (pass == 1 ? 21 : 10)) == digits))
        atomicAdd(&s.hist[0][(kZero >> shift) & mask], zeros);
      __syncthreads();
      const uint32_t sums = remote(smem_u32(&s.hist[1][0]), 0);
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t d = threadIdx.x + i * kThreads, by = s.hist[0][d];
        s.hist[0][d] = 0;
        if (!kCluster) s.hist[1][d] = by;
        else if (by) add_remote(sums + 4 * d, by);
      }
      meet();
      if (rank == 0) {  // the digit where the count of smaller keys passes what is still to leave
        uint4 &bins = *reinterpret_cast<uint4 *>(&s.hist[1][4 * threadIdx.x]);
        const uint4 c = bins;
        bins = make_uint4(0, 0, 0, 0);  // (the others add to it again after the meeting below)
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
#pragma unroll
        for (uint32_t w = 0; w < kWarps; ++w) before += w < warp ? s.warp[w] : 0;
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
          if (!kCluster) s.found[pass] = make_uint2(d, before);
          else
            for (uint32_t r = 0; r < blocks; ++r) st_remote2(remote(smem_u32(&s.found[pass]), r), d, before);
        }
      }
      meet();
      digits = (digits << (pass == 2 ? 10 : 11)) | s.found[pass].x;
      below += s.found[pass].y;
    }
    limit = digits;
  }

  int32_t a[8];  // addresses to be placed: the next are on their way while others are
  addresses(run0, a);
  // what leaves of the runs before this warp's
  uint32_t less = 0, equal = 0;
  if (leave) {
    for (uint32_t i0 = run0; i0 < run1; i0 += 128) {
      uint32_t k[4];
      four(i0 + 4 * lane, k);
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) less += k[j] < limit, equal += k[j] == limit;
    }
    less = __reduce_add_sync(0xffffffffu, less), equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane < blocks) {  // to every block
      if (kCluster) st_remote2(remote(smem_u32(&s.sums[warp][rank]), lane), less, equal);
      else s.sums[warp][0] = make_uint2(less, equal);
    }
    meet();
    less = equal = 0;
    for (uint32_t i = lane; i < warp * blocks + rank; i += 32) {
      const uint2 x = s.sums[i / blocks][i % blocks];
      less += x.x, equal += x.y;
    }
    less = __reduce_add_sync(0xffffffffu, less), equal = __reduce_add_sync(0xffffffffu, equal);
  }
  const uint32_t ties = leave - below;  // equal keys that leave: the first ones
  int32_t *kept = p.kept + (uint64_t)req * p.budget, *dropped = p.dropped + (uint64_t)req * p.dropped_room;
  const uint32_t before = (1u << lane) - 1;
  uint32_t gone = less + (equal < ties ? equal : ties);  // what leaves of the places before these
  for (uint32_t i0 = run0; i0 < run1; i0 += 256) {
    int32_t now[8];
    uint32_t leaves[8];
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) now[j] = a[j];
    addresses(i0 + 256, a);
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) {
      const uint32_t i = i0 + 32 * j + lane;
      uint32_t k = kStays;
      if (leave && i < run1) k = p.cached ? mine[i - run0] : key_at(i, score(now[j]));
      leaves[j] = __ballot_sync(0xffffffffu, k < limit);
      const uint32_t same = __ballot_sync(0xffffffffu, k == limit);
      if (same) {  // (the first of them, so many as may)
        const uint32_t may = equal < ties ? ties - equal : 0;
        leaves[j] |= __ballot_sync(0xffffffffu, k == limit && __popc(same & before) < may);
        equal += __popc(same);
      }
    }
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) {
      const uint32_t i = i0 + 32 * j + lane, at = gone + __popc(leaves[j] & before);
      if (i < run1) {
        if (leaves[j] >> lane & 1) dropped[at] = now[j];
        else kept[i - at] = now[j];
      }
      gone += __popc(leaves[j]);
    }
  }
  for (uint32_t i = n - leave + rank * kThreads + threadIdx.x; i < p.budget; i += blocks * kThreads) kept[i] = -1;
  for (uint32_t i = leave + rank * kThreads + threadIdx.x; i < p.dropped_room; i += blocks * kThreads) dropped[i] = -1;
}

bool aligned4(const void *p) { return ((uintptr_t)p & 3) == 0; }

// Whether n 4-byte words at a and m at b share any.
bool share(const void *a, uint64_t n, const void *b, uint64_t m) {
  return n && m && (uintptr_t)a < (uintptr_t)b + 4 * m && (uintptr_t)b < (uintptr_t)a + 4 * n;
}

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
  // (A list's blocks write their places while others still read theirs: no output lies in an input.)
  const uint64_t n_kept = (uint64_t)n_req * budget, n_dropped = (uint64_t)n_req * p.dropped_room;
  const struct { const void *at; uint64_t n; } inputs[] = {{address, (uint64_t)n_req * longest}, {length, n_req}, {scores, n_scores}};
  for (const auto &in : inputs)
    if (share(kept, n_kept, in.at, in.n) || share(dropped, n_dropped, in.at, in.n)) return ULA_ERR_INVALID_ARG;
  if (share(kept, n_kept, dropped, n_dropped)) return ULA_ERR_INVALID_ARG;
  // 2,048 places a block, 4 a thread, before another joins: a block's passes over its keys then take less
  // than a meeting.  (The case at the top with clusters of 4: 40 us, with 8 39, when it was compared.)
  uint32_t cluster = 1;
  while (cluster < kMostCluster && longest > cluster * 2048) cluster *= 2;
  if ((uint64_t)n_req * cluster > 0x7fffffffull) return ULA_ERR_INVALID_ARG;
  const uint32_t run = run_of(longest, cluster);
  // (32 lists of up to 393,216 addresses: 124 us; of 400,000, whose scores are gathered again in every pass, 180)
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
