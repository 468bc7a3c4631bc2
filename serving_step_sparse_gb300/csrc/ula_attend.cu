// Attention over the cache's FP8 rows (ula_rows_attend).
//
// For a query token and its entries e, with codes c (e4m3), block scales s, rope k and a
// head's query (q_0..q_3 latent blocks, q_r rope):
//   z[e] = c0 * (sum_b s_b(e) <q_b, c_b(e)> + <q_r, k(e)>),  p = exp2(z - m),
//   out  = sum_e p[e] s_b(e) c_b(e) / sum_e p[e]   (channels of block b),
// with c0 = softmax_scale * log2(e) and m a running maximum.
//
// Both products run on the tensor cores with the rows transposed into the M dimension:
// S^T[128 rows][heads] = C_b Q_b^T for each block b (and the rope part), and
// O^T[128 channels][heads] += C_b^T P_b^T.  So any head count fits in N without waste, a
// thread of the softmax owns one row (its scales are four registers), and the codes serve
// both products from one bf16 copy in shared memory (K-major for the first, MN-major for
// the second).  A code is exact in bf16 and its scale multiplies fp32 accumulators, so the
// logits are as exact as fp32 sums; the probabilities times the scales enter the second
// product in bf16 (up to 2^-8 relative on each, which averages out over the rows; bf16 and not
// f16 since scales may span many orders).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <atomic>
#include <map>
#include <mutex>
#include <utility>

#include "ula.h"
#include "ula_tc.cuh"

using namespace ula_tc;

namespace {

__device__ uint32_t g_late;  // warps whose waits ran out, in all launches so far

constexpr uint32_t kTile = 128;                      // rows per tile
constexpr uint32_t kGroupBytes = kTile * 128;        // 64 channels of a tile's rows, bf16
constexpr uint32_t kGroups = 9;                      // 8 of latents, 1 of rope
constexpr uint32_t kWarps = 8;                       // compute warps; then an issuing one, two loading, an issuing one
constexpr uint32_t kThreads = (kWarps + 4) * 32;     // (registers move between groups of 4 warps)
// Launched with 168 registers a thread: 3 * 168 = 2 * 216 + 72.
constexpr uint32_t kRegsCompute = 216, kRegsIssue = 72;
constexpr uint32_t kLoaders = 2;                     // loading warps, 64 rows each
constexpr uint32_t kSlots = kTile / (4 * kWarps / 2);  // rows per lane of the widening
constexpr uint32_t kMostCluster = 8;                  // (the portable size)
constexpr uint32_t kColS = 256;                      // TMEM: O^T in columns 0.., S^T from here

struct AttendParams {
  ula_attend_args a;
  // An item is a query token and a tile of heads.  Block c takes items c, c + blocks, ... whole, as
  // many rounds as there are for all blocks; of the remaining items' tiles the first `sharers`
  // blocks (all, or as many as there are tiles) take [c * rest / sharers, (c + 1) * rest / sharers).
  unsigned long long rest;   // tiles of the remaining items
  uint32_t blocks, rounds, sharers;
  uint32_t tiles;            // tiles per item
  uint32_t head_tiles;
  uint32_t keys;             // entries per query token, own rows included
  uint32_t cluster;          // blocks of a cluster (one item each), or 1
  float c0;
  uint32_t hold;             // (test hook) an mbarrier whose phases never end; kBars: none
  // A tree (ula_rows_attend_tree): own row j stands for node j of the request's tree.  A list's columns
  // (a.heads) are one node's query heads or, where the tree shares the list, all nodes'; a.n_q is
  // the number of lists of a request.
  const int32_t *parent;     // [n_req][nodes]
  uint32_t nodes, node_heads;
  float *part_out;           // [2 * blocks][NH][512]: unfinished items' results, normalised
  float *part_lse;           // [2 * blocks][NH]: their log2 sums
};

// ---------------------------------------------------------------- the kernel

// mbarriers.  Full + b: block b of the tile stands in shared memory (4: the rope); S + b: S_b^T in
// TMEM; Drained: block 1's S^T has been read; P: P_0, and P_1 to P_3, stand in shared memory; PV + b:
// O_b^T is up to date and block b's codes are free; X: exchange in a column group; Place: the rows'
// addresses stand; Scale: their scales; End: a warp's products have ended.
enum {
  kBarFull = 0, kBarS = 5, kBarDrained = 10, kBarP = 11, kBarPV = 13, kBarX = 17, kBarPlace = 19, kBarScale = 20, kBarEnd = 21,
  kBars = ULA_DEBUG_BARRIERS
};

template <uint32_t NH>
struct Shared {
  static constexpr uint32_t q = 0;                            // [9][NH][128 B]
  static constexpr uint32_t k = kGroups * NH * 128;           // [9][128][128 B]
  static constexpr uint32_t scale = k + kGroups * kGroupBytes;  // [128][4] the rows' scales
  static constexpr uint32_t place = scale + kTile * 16;       // [2][128] the rows' addresses, 0: no row
  static constexpr uint32_t sees = place + 2 * kTile * 8;     // [2][128] (a tree) which columns see them
  static constexpr uint32_t top = sees + 2 * kTile * 8;       // [NH][4] tile maxima (then sums) by quadrant
  static constexpr uint32_t bars = top + NH * 16;
  static constexpr uint32_t words = bars + 24 * 8;            // TMEM address; first remaining item, its tile; tiles in all
  static constexpr uint32_t bytes = words + 16 + 1024;        // (+ alignment of the base)
};

// The tiles of a block, in item order.
struct Place {
  uint32_t item, tile;       // the tile's item and place in it
  uint32_t token, req, qi, h0;
};

template <uint32_t NH>
__device__ __forceinline__ void decode(const AttendParams &p, Place &w) {
  w.token = w.item / p.head_tiles;
  w.h0 = (w.item - w.token * p.head_tiles) * NH;
  w.req = w.token / p.a.n_q;
  w.qi = w.token - w.req * p.a.n_q;
}

template <uint32_t NH>
__device__ __forceinline__ void step(const AttendParams &p, Place &w, const volatile uint32_t *words) {
  if (++w.tile == p.tiles) {
    w.tile = 0;
    const uint32_t whole = p.rounds * p.blocks;  // items
    if (w.item >= whole) {
      ++w.item;
    } else if ((w.item += p.blocks) >= whole) {
      w.item = words[1], w.tile = words[2];
    }
    decode<NH>(p, w);
  }
}

// Entry e of a tile's query token as it stands in memory (0 past the list).  What it means is
// worked out when the rows are fetched: a comparison here would wait for the load.
__device__ __forceinline__ int32_t entry_of(const AttendParams &p, const Place &at, uint32_t e) {
  return e < p.a.k ? __ldg(p.a.entry_row + (uint64_t)at.token * p.a.k + e) : 0;
}

// Its row (0: none).  Entries behind the list stand for the request's own rows (of a tree: all of
// them; which node sees which is masked after the products).
template <bool kTree>
__device__ __forceinline__ uint64_t row_of(const AttendParams &p, const Place &at, uint32_t e, int32_t u) {
  if (e < p.a.k)
    return u >= 0 && (uint32_t)u < p.a.n_rows ? (uint64_t)p.a.rows + (uint64_t)u * ULA_ROW_BYTES : 0;
  const uint32_t j = e - p.a.k;
  if (e >= p.keys || (!kTree && j > at.qi)) return 0;
  return (uint64_t)p.a.own_rows + at.req * p.a.own_req_stride + j * p.a.own_tok_stride;
}

// The join of partial results of one query head: 4 channels, a running maximum over batches
// of parts (whose loads are all in flight together).
struct Joined {
  float m = -INFINITY, total = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  template <uint32_t N>
  __device__ __forceinline__ void add(const float (&l)[N], const float4 (&o)[N]) {
    float top = m;
#pragma unroll
    for (uint32_t k = 0; k < N; ++k) top = fmaxf(top, l[k]);
    const float ref = top == -INFINITY ? 0.f : top, old = ex2(m - ref);
    m = top;
    total *= old, acc.x *= old, acc.y *= old, acc.z *= old, acc.w *= old;
#pragma unroll
    for (uint32_t k = 0; k < N; ++k) {
      const float f = ex2(l[k] - ref);
      total += f;
      acc.x += f * o[k].x, acc.y += f * o[k].y, acc.z += f * o[k].z, acc.w += f * o[k].w;
    }
  }
  __device__ __forceinline__ void write(const ula_attend_args &a, uint64_t row, uint32_t c) const {
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const uint2 r = make_uint2(bf16x2(acc.x * inv, acc.y * inv), bf16x2(acc.z * inv, acc.w * inv));
    reinterpret_cast<uint2 *>((__nv_bfloat16 *)a.out + row * ULA_ROW_LATENT)[c] = r;
    if (a.lse && c == 0) a.lse[row] = ((m == -INFINITY ? 0.f : m) + log2f(total)) * 0.693147180559945309f;
  }
};

// The bits of the ancestors of a tree's nodes, each node's own among them: lane l gets node l's and
// node (l + 32)'s.  By doubling: after n steps a node has its ancestors up to 2^n - 1 levels up.
__device__ __forceinline__ void ancestors(const int32_t *parent, uint32_t nodes, uint32_t lane, uint64_t (&seen)[2]) {
  int32_t up[2];
#pragma unroll
  for (uint32_t i = 0; i < 2; ++i) {
    const int32_t node = (int32_t)(lane + 32 * i);
    up[i] = (uint32_t)node < nodes ? __ldg(parent + node) : -1;
    if (up[i] < 0 || up[i] >= node) up[i] = -1;  // (none but an earlier node is a parent)
    seen[i] = 1ull << node;
  }
  for (uint32_t reach = 1; reach < nodes; reach *= 2) {
    uint64_t more[2];
    int32_t next[2];
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) {
      const uint64_t s0 = __shfl_sync(0xffffffffu, seen[0], up[i] & 31), s1 = __shfl_sync(0xffffffffu, seen[1], up[i] & 31);
      const int32_t n0 = __shfl_sync(0xffffffffu, up[0], up[i] & 31), n1 = __shfl_sync(0xffffffffu, up[1], up[i] & 31);
      more[i] = up[i] < 0 ? 0 : up[i] < 32 ? s0 : s1;
      next[i] = up[i] < 0 ? -1 : up[i] < 32 ? n0 : n1;
    }
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) seen[i] |= more[i], up[i] = next[i];
  }
}

// Which columns (nodes and heads, of the item's NH) see a tile's rows e and e + 32: a bit each, as their nodes
// or ancestors of them; all for the list's rows.
template <uint32_t NH>
__device__ __forceinline__ void see_tree(const AttendParams &p, const Place &w, uint32_t e, uint64_t (&sees)[2]) {
  uint64_t seen[2];
  ancestors(p.parent + (uint64_t)w.req * p.nodes, p.nodes, threadIdx.x & 31, seen);
  uint32_t node = w.h0 / p.node_heads, left = (node + 1) * p.node_heads - w.h0;
  node += w.qi;
  sees[0] = sees[1] = 0;
#pragma unroll 1
  for (uint32_t h = 0; h < NH; ++node, left = p.node_heads) {  // (by runs of a node's heads)
    const uint64_t s0 = __shfl_sync(0xffffffffu, seen[0], node & 31), s1 = __shfl_sync(0xffffffffu, seen[1], node & 31);
    const uint64_t mask = node < 32 ? s0 : s1;
    const uint32_t n = left < NH - h ? left : NH - h;
    const uint64_t run = (n < 64 ? (1ull << n) - 1 : ~0ull) << h;
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) {
      const uint32_t at = e + 32 * i, j = at - p.a.k;
      if (at < p.a.k || j >= p.nodes || (mask >> j & 1)) sees[i] |= run;
    }
    h += n;
  }
}

// A row's widened codes without their NaN.  (Any order: the swizzle stays within a row's 128 bytes.)
__device__ __noinline__ void clean_codes(uint8_t *codes) {
#pragma unroll 1
  for (uint32_t i = 0; i < 256; ++i) {
    uint32_t *at = reinterpret_cast<uint32_t *>(codes + (i >> 5) * kGroupBytes) + (i & 31);
    uint32_t two = *at;
    if ((two & 0x7fff0000u) > 0x7f800000u) two &= 0xffffu;
    if ((two & 0x7fffu) > 0x7f80u) two &= 0xffff0000u;
    *at = two;
  }
}

// Persistent: one block per SM, which runs whole items first, then an even share of the rest's
// tiles (an item whose tiles end up in several blocks leaves one partial result in each;
// k_join_parts joins them).  8 compute warps fetch the rows' codes into registers one tile ahead, widen
// them to bf16 in shared memory and run the softmax; two warps look the rows up and copy
// their scales and rope channels; two issue the products.  Compute warp w reads TMEM lanes
// (rows) 32 (w % 4).. and the heads of column group w / 4.
//
// What bounds it: the one tile in shared memory (queries 72 KB, tile 144 KB at 64 heads) makes
// widening, S^T, softmax and O^T of a tile follow each other, some 9,000 clocks a tile, of
// which its 68 products take 3,500 (their operands' bytes from shared memory, not their
// arithmetic), its rows 2,700 (82 KB at the 30 B a clock that an SM exchanges with L2, in either
// direction) and the conversions 1,600.  96 tokens, 2,048 + 3 rows, with the join: 128 heads
// 119 us (0.46 PFLOP/s), 64 heads 72 us, and 15.5 us for 8 tokens of 64 heads.  (When they were
// compared, before the loads were spread, 16 compute warps of half the registers took 12, 5 and
// 0.4 us more than 8.)
//
// Shared memory holds one tile, and the tile's own parts make room for P (P_b = p * s_b,
// 16 KB): P_0 takes the rope's place; after O_0 has read block 0's codes, P_1 and P_3 take
// theirs and P_2 the rope's.  So the next tile's blocks are widened in the order 1, 2, then 0
// and 3, as O_1, O_2 and O_3 finish, beside the rest of the products; their codes wait in
// registers, and the rope is copied in after O_2.
//
// kCluster: the tiles of one item spread over the blocks of a cluster, which join their
// results through each other's shared memory (no second kernel, no trip through L2).
// kTree: a column is a node and a head, and own rows are masked by the nodes' ancestors.
template <uint32_t NH, bool kCluster, bool kTree>
__global__ void __launch_bounds__(kThreads, 1)
k_attend(const __grid_constant__ AttendParams p) {
  extern __shared__ uint8_t raw_smem[];
  using L = Shared<NH>;
  constexpr int HG = NH / (kWarps / 4);  // heads per column group
  const uint32_t base = (smem_u32(raw_smem) + 1023u) & ~1023u;
  uint8_t *sm = raw_smem + (base - smem_u32(raw_smem));
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](uint32_t i) { return base + L::bars + 8 * i; };
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < 5; ++i) {
      mbar_init(bar(kBarFull + i), i < 4 ? kWarps / 2 : kLoaders);
      mbar_init(bar(kBarS + i), 1);
    }
    mbar_init(bar(kBarPlace), kLoaders), mbar_init(bar(kBarScale), kLoaders * 32);
    mbar_init(bar(kBarDrained), kWarps);
    mbar_init(bar(kBarP), kWarps), mbar_init(bar(kBarP + 1), kWarps);
    for (uint32_t i = 0; i < 4; ++i) mbar_init(bar(kBarPV + i), 1);
    for (uint32_t i = 0; i < kWarps / 4; ++i) mbar_init(bar(kBarX + i), 4);
    mbar_init(bar(kBarEnd), 1), mbar_init(bar(kBarEnd + 1), 1);
    if (p.hold < kBars) {
      asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar(p.hold)) : "memory");
      mbar_init(bar(p.hold), 1u << 19);  // (more arrivals than a launch makes)
    }
    fence_async_smem();
  }
  // (an address read before its time, after a wait that ran out, is no address)
  if (threadIdx.x < 2 * kTile) reinterpret_cast<uint64_t *>(sm + L::place)[threadIdx.x] = 0;
  if (warp == kWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + L::words) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(sm + L::words);
  if (threadIdx.x == 32) {  // where its share of the remaining items (a cluster's: of its item) starts, and its tiles in all
    uint32_t item, tile, count;
    if (kCluster) {
      item = blockIdx.x / p.cluster;
      const uint32_t rank = blockIdx.x - item * p.cluster;
      tile = rank * p.tiles / p.cluster;
      count = (rank + 1) * p.tiles / p.cluster - tile;
    } else {
      const unsigned long long first = p.rest * blockIdx.x / p.sharers;
      item = (uint32_t)(first / p.tiles), tile = (uint32_t)(first - (unsigned long long)item * p.tiles);
      item += p.rounds * p.blocks;
      count = p.rounds * p.tiles;
      if (blockIdx.x < p.sharers) count += (uint32_t)(p.rest * (blockIdx.x + 1) / p.sharers - first);
    }
    words[1] = item, words[2] = tile, words[3] = count;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, words[0], 0);
  // (launched while the kernel before it ends: nothing above touches memory that it may write)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Place w;
  w.item = p.rounds ? blockIdx.x : words[1], w.tile = p.rounds ? 0 : words[2];
  const uint32_t count = words[3];
  const uint32_t sk = base + L::k;
  // all threads of the cluster; those that have given up on a wait as well
  auto meet = [] {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  };

  bool ok = true;  // false once a wait has run out
  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == kWarps || warp == kWarps + 1 + kLoaders) {
      // ---- the products, issued by two warps.  A warp waits as one and one elected lane
      // issues, so that the operands' descriptors stay in uniform registers.  A wait is held
      // up until the warp's products before it have left the queue (155 clocks each with the
      // queue run dry), so the warps take the S_b^T in turn: 36 products of N = 64 in 1,900
      // clocks, which is what their operands take, instead of 2,990.  For the same reason a
      // wait that has run out does not leave the loop (the compiler would then take all that
      // follows for divergent): the rest goes unwaited for, and is reported at the end.
      // D fp32, A and B bf16; M = 128, N = NH; for O^T both operands are MN-major
      constexpr uint32_t kIdS = (1u << 4) | (1u << 7) | (1u << 10) | ((NH >> 3) << 17) | ((kTile >> 4) << 24);
      constexpr uint32_t kIdO = kIdS | (1u << 15) | (1u << 16);
      uint64_t k_rows = operand(sk, 16), k_channels = operand(sk, kGroupBytes), q_rows = operand(base + L::q, 16);
      // S_b^T; the rope's part (4) goes to block 1's columns
      auto issue_s = [&](uint32_t b) {
        tc_fence_after();
        const uint32_t d = tmem + kColS + (b == 4 ? 1 : b) * NH;
        const uint64_t da = k_rows + b * (2 * kGroupBytes >> 4), db = q_rows + b * (2 * NH * 128 >> 4);
        if (elect_one()) {
#pragma unroll
          for (uint32_t s = 0; s < (b == 4 ? 4 : 8); ++s)
            mma_bf16(d, da + (s >> 2) * (kGroupBytes >> 4) + (s & 3) * 2, db + (s >> 2) * (NH * 128 >> 4) + (s & 3) * 2, kIdS, s != 0);
          mma_commit(bar(kBarS + b));
        }
        __syncwarp();
      };
      if (warp == kWarps) {
        uint32_t tile = w.tile;
        bool fresh = true;
        for (uint32_t n = 0; n < count; ++n) {
          const uint32_t par = n & 1;
          // (new to the compiler in every tile: it would keep 68 descriptors in registers otherwise)
          asm volatile("" : "+l"(k_rows), "+l"(k_channels), "+l"(q_rows));
          ok = ok && warp_wait(bar(kBarFull + 1), par, bar(kBarFull + 2), par);  // (every warp's queries)
          issue_s(1);
          ok = ok && warp_wait(bar(kBarFull), par);
          issue_s(0);
          ok = ok && warp_wait(bar(kBarP), par);
          tc_fence_after();
#pragma unroll
          for (uint32_t b = 0; b < 4; ++b) {  // O_b^T
            if (b == 1) {
              ok = ok && warp_wait(bar(kBarP + 1), par);
              tc_fence_after();
            }
            const uint64_t da = k_channels + b * (2 * kGroupBytes >> 4);
            const uint64_t db = k_channels + (b == 1 ? 0 : b == 3 ? 1 : 8) * (kGroupBytes >> 4);
            if (elect_one()) {
#pragma unroll
              for (uint32_t s = 0; s < 8; ++s) mma_bf16(tmem + b * NH, da + s * 128, db + s * 128, kIdO, s != 0 || !fresh);
              mma_commit(bar(kBarPV + b));
            }
            __syncwarp();
          }
          fresh = false;
          if (++tile == p.tiles) tile = n + 1 == p.rounds * p.tiles ? words[2] : 0, fresh = true;
        }
      } else {
        for (uint32_t n = 0; n < count; ++n) {
          const uint32_t par = n & 1;
          asm volatile("" : "+l"(k_rows), "+l"(q_rows));
          ok = ok && warp_wait(bar(kBarFull + 1), par, bar(kBarFull + 2), par);  // (every warp's queries)
          issue_s(2);
          ok = ok && warp_wait(bar(kBarFull + 3), par);
          issue_s(3);
          ok = ok && warp_wait(bar(kBarFull + 4), par, bar(kBarDrained), par);  // (block 1's columns have been read)
          issue_s(4);
        }
      }
      const uint32_t end = bar(kBarEnd + (warp == kWarps ? 0 : 1));
      bool ended = true;
      if (elect_one()) {  // every product has ended before the block's TMEM goes
        mma_commit(end);
        ended = mbar_wait(end, 0);
      }
      ok = __all_sync(0xffffffffu, ended) && ok;
    } else if (warp <= kWarps + kLoaders) {
      // ---- this warp's 64 rows of every tile: their addresses, one tile ahead (two a lane),
      // their scales, and their rope channels straight to where the products read them
      decode<NH>(p, w);
      const uint32_t r0 = (warp - kWarps - 1) * 64;
      int32_t u[2];
      auto fetch_entries = [&]() {
        u[0] = entry_of(p, w, w.tile * kTile + r0 + lane);
        u[1] = entry_of(p, w, w.tile * kTile + r0 + lane + 32);
      };
      auto place_rows = [&](uint32_t par) {
        uint64_t *place = reinterpret_cast<uint64_t *>(sm + L::place) + par * kTile + r0;
        uint64_t *seen = reinterpret_cast<uint64_t *>(sm + L::sees) + par * kTile + r0;
        const uint32_t e = w.tile * kTile + r0 + lane;
        uint64_t sees[2] = {~0ull, ~0ull};
        if (kTree && (w.tile + 1) * kTile > p.a.k) see_tree<NH>(p, w, e, sees);  // (the tile holds nodes' rows)
#pragma unroll
        for (uint32_t j = 0; j < 2; ++j) {
          const uint64_t row = row_of<kTree>(p, w, e + 32 * j, u[j]);
          place[lane + 32 * j] = row;
          if (kTree) seen[lane + 32 * j] = row ? sees[j] : 0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPlace));
      };
      fetch_entries();
      place_rows(0);
      for (uint32_t n = 0; n < count; ++n) {
        const uint32_t par = n & 1, prev = par ^ 1;
        const uint64_t *place = reinterpret_cast<const uint64_t *>(sm + L::place) + par * kTile + r0;
        if (n + 1 < count) {
          step<NH>(p, w, words);
          fetch_entries();
        }
        if (n && !(ok = warp_wait(bar(kBarPV + 1), prev))) break;
#pragma unroll
        for (uint32_t j = 0; j < 2; ++j) {
          const uint64_t row = place[lane + 32 * j];
          copy16(base + L::scale + (r0 + lane + 32 * j) * 16, (const void *)(row ? row + ULA_ROW_LATENT : (uint64_t)p.a.q), row ? 16 : 0);
        }
        copy_arrive(bar(kBarScale));
        if (n && !(ok = warp_wait(bar(kBarPV + 2), prev))) break;
#pragma unroll
        for (uint32_t i = 0; i < 16; ++i) {
          const uint32_t r = r0 + 4 * i + (lane >> 3), ch = lane & 7;
          const uint64_t row = place[4 * i + (lane >> 3)];
          copy16(sk + 8 * kGroupBytes + r * 128 + ((ch ^ (r & 7)) << 4),
                 (const void *)(row ? row + ULA_ROW_LATENT + 16 + ch * 16 : (uint64_t)p.a.q), row ? 16 : 0);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarFull + 4));
        // The next addresses only once every compute warp has this tile's: a second arrival of
        // one loading warp may not stand for the first of the other.
        if (n + 1 < count) {
          ok = warp_wait(bar(kBarFull + 1), par);
          if (!(ok = ok && warp_wait(bar(kBarFull + 2), par))) break;
          place_rows(prev);
          // into L2 ahead of the loads: 2 % of 128 heads' time when it came in.  (Not for a block's first
          // tile, whose loads follow at once: that took 1.2 us of one request's 9.6 more.)
          const uint64_t *ahead = reinterpret_cast<const uint64_t *>(sm + L::place) + prev * kTile + r0;
#pragma unroll
          for (uint32_t j = 0; j < 2; ++j)
            if (ahead[lane + 32 * j]) prefetch((const void *)ahead[lane + 32 * j], ULA_ROW_BYTES);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
    if (kCluster) meet();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsCompute));
    decode<NH>(p, w);
    const uint32_t quad = warp & 3, grp = warp >> 2;
    const uint32_t lanes = tmem + (quad << 21);  // TMEM lane 32 * quad
    const uint32_t mine = 32 * quad + lane;      // this thread's row in the softmax
    // widening: the first half of the warps does blocks 1 and 0, the other 2 and 3; a lane rows r0,
    // r0 + 4, ..., 16 channels ch of a block.  16-byte accesses are served by quarters of a
    // warp: a quarter loads 128 bytes of one row, and stores to 8 different chunks of its
    // swizzled row, since lanes of the second half store their second chunk first.
    const bool second = warp >= kWarps / 2;
    const uint32_t r0 = 4 * kSlots * (warp & (kWarps / 2 - 1)) + (lane >> 3), ch = lane & 7;
    float *top = reinterpret_cast<float *>(sm + L::top) + grp * HG * 4;
    uint32_t xph = 0;
    auto exchange = [&]() -> bool {  // the four warps of a column group
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarX + grp));
      const bool met = warp_wait(bar(kBarX + grp), xph);
      xph ^= 1;
      return met;
    };
    auto hand_over = [&](uint32_t b) {
      fence_async_smem();
      tc_fence_before();  // (this warp's TMEM accesses so far)
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
    };
    const uint32_t block1 = second ? 2 : 1, block2 = second ? 3 : 0;
    // Half of this thread's codes of one block, of tile n's rows.  The next tile's come in four such
    // pieces of 16 KB, apart from each other: more than some 28 KB of loads in flight stop the
    // load/store unit for the shared memory's accesses as well (128 heads, 2,051 rows, when it came in:
    // 125 us; 135 in pieces of 24, 24 and 16 KB, 141 in one of 64).
    auto fetch = [&](uint4 (&raw)[kSlots], uint32_t n, uint32_t block, uint32_t half) {
      const uint64_t *place = reinterpret_cast<const uint64_t *>(sm + L::place) + (n & 1) * kTile;
#pragma unroll
      for (uint32_t j = half * (kSlots / 2); j < (half + 1) * (kSlots / 2); ++j) {
        const uint64_t row = place[r0 + 4 * j];
        raw[j] = make_uint4(0, 0, 0, 0);
        if (row) raw[j] = __ldg(reinterpret_cast<const uint4 *>(row + block * 128 + ch * 16));
      }
    };
    auto widen = [&](const uint4 (&raw)[kSlots], uint32_t b) {
#pragma unroll
      for (uint32_t j = 0; j < kSlots; ++j) {
        const uint32_t r = r0 + 4 * j, x = r & 7;
        const uint4 v = raw[j];
        uint8_t *at = sm + L::k + (2 * b + (ch >> 2)) * kGroupBytes + r * 128;
        const bool up = ch & 4;
        const uint32_t c = 2 * (ch & 3) + (up ? 1 : 0);
        const uint32_t p0 = up ? v.z : v.x, p1 = up ? v.w : v.y, q0 = up ? v.x : v.z, q1 = up ? v.y : v.w;
        *reinterpret_cast<uint4 *>(at + ((c ^ x) << 4)) =
            make_uint4(codes_to_bf16(p0), codes_to_bf16(p0 >> 16), codes_to_bf16(p1), codes_to_bf16(p1 >> 16));
        *reinterpret_cast<uint4 *>(at + ((c ^ 1 ^ x) << 4)) =
            make_uint4(codes_to_bf16(q0), codes_to_bf16(q0 >> 16), codes_to_bf16(q1), codes_to_bf16(q1 >> 16));
      }
      hand_over(kBarFull + b);
    };

    uint4 raw1[kSlots], raw2[kSlots];
    float sum[HG], ref = -INFINITY;  // this row's sums; lane h: head h's running maximum
    bool start = true;               // the first tile of a piece
    uint32_t first_tile = w.tile;
    // the queries of w's item
    auto load_queries = [&]() {
      const __nv_bfloat16 *q = (const __nv_bfloat16 *)p.a.q + w.req * p.a.q_req_stride + w.qi * p.a.q_tok_stride;
      if (kTree) {  // (a warp a column, whose node and head are worked out once)
        for (uint32_t h = warp; h < NH; h += kWarps) {
          const bool in = w.h0 + h < p.a.heads;
          const uint32_t node = (w.h0 + h) / p.node_heads;
          const __nv_bfloat16 *src = q + (in ? node * p.a.q_tok_stride + (w.h0 + h - node * p.node_heads) * p.a.q_head_stride : 0);
          const uint32_t dst = base + L::q + (lane >> 3) * (NH * 128) + h * 128 + (((lane & 7) ^ (h & 7)) << 4);
          copy16(dst, src + lane * 8, in ? 16 : 0);
          copy16(dst + 4 * NH * 128, src + (32 + lane) * 8, in ? 16 : 0);
          if (lane < 8) copy16(dst + 8 * NH * 128, src + (64 + lane) * 8, in ? 16 : 0);
        }
      }
      for (uint32_t i = threadIdx.x; !kTree && i < NH * 72; i += kWarps * 32) {
        const uint32_t h = i / 72, c = i - h * 72;
        const uint32_t dst = base + L::q + (c >> 3) * (NH * 128) + h * 128 + (((c & 7) ^ (h & 7)) << 4);
        const bool in = w.h0 + h < p.a.heads;
        const __nv_bfloat16 *src = q + (in ? (w.h0 + h) * p.a.q_head_stride + c * 8 : 0);
        copy16(dst, src, in ? 16 : 0);
      }
    };
    load_queries();  // (while the first rows are looked up)
    ok = warp_wait(bar(kBarPlace), 0);
    if (ok) {
      fetch(raw1, 0, block1, 0), fetch(raw1, 0, block1, 1);
      fetch(raw2, 0, block2, 0), fetch(raw2, 0, block2, 1);
    }
    for (uint32_t n = 0; n < count && ok; ++n) {
      const uint32_t par = n & 1;
      if (start) {
        first_tile = w.tile;
#pragma unroll
        for (int h = 0; h < HG; ++h) sum[h] = 0.f;
        ref = -INFINITY;
        if (n) load_queries();  // (the products that read the previous item's have ended)
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
      // ---- widen the tile, block by block as there is room (in a loop, since two copies of this
      // code fall out of the instruction caches: 3 % more)
#pragma unroll 1
      for (uint32_t half = 0; half < 2; ++half) {
        if (n && !(ok = warp_wait(bar(kBarPV + (half ? 3 : block1)), par ^ 1))) break;
        widen(raw1, half ? block2 : block1);
#pragma unroll
        for (uint32_t j = 0; j < kSlots; ++j) raw1[j] = raw2[j];
      }
      if (!ok) break;
      // this row's scales, and whether there is a row; block 1's product (and the next tile's rows)
      const bool more = n + 1 < count;
      ok = more ? warp_wait(bar(kBarScale), par, bar(kBarS + 1), par, bar(kBarPlace), par ^ 1) : warp_wait(bar(kBarScale), par, bar(kBarS + 1), par);
      if (!ok) break;
      float4 scale = *reinterpret_cast<const float4 *>(sm + L::scale + mine * 16);
      const bool present = reinterpret_cast<const uint64_t *>(sm + L::place)[par * kTile + mine] != 0;

      // ---- logits in units of log2, this thread's row and HG heads: the scales carry c0.
      // Block 1's part comes first, so that the rope's product can take its columns.
      float z[HG];
      {
        float v[HG];
        tc_fence_after();
        tmem_ld<HG>(lanes + kColS + NH + grp * HG, v);
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarDrained));
        const float s = scale.y * p.c0;
#pragma unroll
        for (int h = 0; h < HG; h += 2) mul2(z[h], z[h + 1], s, v[h], v[h + 1]);
      }
      if (more) fetch(raw1, n + 1, block1, 0);
      {
        float v[HG], x[HG];
        if (!(ok = warp_wait(bar(kBarS + 2), par, bar(kBarS), par))) break;
        tc_fence_after();
        tmem_ld<HG>(lanes + kColS + 2 * NH + grp * HG, v);
        tmem_ld<HG>(lanes + kColS + grp * HG, x);
        tc_wait_ld();
        float s = scale.z * p.c0, t = scale.x * p.c0;
#pragma unroll
        for (int h = 0; h < HG; h += 2) {
          fma2(z[h], z[h + 1], s, v[h], v[h + 1]);
          fma2(z[h], z[h + 1], t, x[h], x[h + 1]);
        }
        if (!(ok = warp_wait(bar(kBarS + 3), par, bar(kBarS + 4), par))) break;
        tc_fence_after();
        tmem_ld<HG>(lanes + kColS + 3 * NH + grp * HG, v);
        tmem_ld<HG>(lanes + kColS + NH + grp * HG, x);
        tc_wait_ld();
        s = scale.w * p.c0, t = p.c0;
#pragma unroll
        for (int h = 0; h < HG; h += 2) {
          fma2(z[h], z[h + 1], s, v[h], v[h + 1]);
          fma2(z[h], z[h + 1], t, x[h], x[h + 1]);
        }
      }

      // A row that is not there gets logits of -inf, whatever the products say: its zeros times a NaN
      // or an infinity of the query are NaN.
      if (!kTree && !__all_sync(0xffffffffu, present)) {
#pragma unroll
        for (int h = 0; h < HG; ++h) z[h] = present ? z[h] : -INFINITY;
      }
      // Of a tree's own rows a column (a node and a head) sees its node's and its ancestors'.  The loading warps
      // have worked out which: here, unrolled over the columns, that took 11 % of the whole, as it runs once an
      // item and its instructions are fetched each time.
      if (kTree) {
        const uint32_t sees = (uint32_t)(reinterpret_cast<const uint64_t *>(sm + L::sees)[par * kTile + mine] >> (grp * HG));
        constexpr uint32_t kAll = HG < 32 ? (1u << (HG & 31)) - 1 : 0xffffffffu;
        // A row that some see and others do not is in the products of both, with a probability of 0 for the
        // latter, so what it holds must be finite: one with a NaN among its codes (all its logits are NaN) or a
        // scale that is not finite gives NaN to those who see it here, and goes on with codes and scales that
        // are.  (Both threads of a row may write its codes: the same values.)
        // (Asked in every tile: behind a test for tiles with own rows it took 2.5 % more of the whole.)
        const bool bad = present && w.tile * kTile + mine >= p.a.k &&
                         (z[0] != z[0] || !(isfinite(scale.x) && isfinite(scale.y) && isfinite(scale.z) && isfinite(scale.w)));
        if (__any_sync(0xffffffffu, bad)) {
          bool all = bad;
#pragma unroll
          for (int h = 1; h < HG; ++h) all = all && z[h] != z[h];  // (not a NaN of the first column's query alone)
          if (bad && !(isfinite(scale.x) && isfinite(scale.y) && isfinite(scale.z) && isfinite(scale.w))) all = true;
          if (all) {
            scale = make_float4(1.f, 1.f, 1.f, 1.f);
            clean_codes(sm + L::k + mine * 128);
          }
#pragma unroll
          for (int h = 0; h < HG; ++h) z[h] = all ? __int_as_float(0x7fffffff) : z[h];
        }
        if (!__all_sync(0xffffffffu, (sees & kAll) == kAll)) {
#pragma unroll
          for (int h = 0; h < HG; ++h) z[h] = sees >> h & 1 ? z[h] : -INFINITY;
        }
      }

      if (more) fetch(raw1, n + 1, block1, 1);
      // ---- running maximum: it moves only when a tile's is more than 8 (a factor of 256)
      // above it, so that O^T is seldom rescaled; p stays below 2^8.  Lane h keeps head h's.
      {
        float t = -INFINITY;
#pragma unroll
        for (int h = 0; h < HG; ++h) {
          const float m = warp_max(z[h]);
          if (lane == (uint32_t)h) t = m;
        }
        if (lane < HG) top[lane * 4 + quad] = t;
      }
      if (!(ok = exchange())) break;
      {
        const float4 t4 = *reinterpret_cast<const float4 *>(top + (lane & (HG - 1)) * 4);
        const float t = fmaxf(fmaxf(t4.x, t4.y), fmaxf(t4.z, t4.w));
        const bool up = t > ref + 8.f;
        const float now = up ? t : ref;
        if (__any_sync(0xffffffffu, up)) {  // (the same in all four warps)
          const float f = up ? ex2(ref - now) : 1.f;
#pragma unroll
          for (int h = 0; h < HG; ++h) sum[h] *= __shfl_sync(0xffffffffu, f, h);
          if (!start) {  // (the products into O^T so far have ended: waited for above)
#pragma unroll 1
            for (uint32_t b = 0; b < 4; ++b) {
#pragma unroll
              for (int c = 0; c < HG; c += 4) {
                float o[4];
                tmem_ld<4>(lanes + b * NH + grp * HG + c, o);
                tc_wait_ld();
#pragma unroll
                for (int h = 0; h < 4; ++h) o[h] *= __shfl_sync(0xffffffffu, f, c + h);
                tmem_st<4>(lanes + b * NH + grp * HG + c, o);
              }
            }
            tc_wait_st();
          }
        }
        ref = now;
        const float m = now == -INFINITY ? 0.f : now;
#pragma unroll
        for (int h = 0; h < HG; ++h) {
          z[h] = ex2(z[h] - __shfl_sync(0xffffffffu, m, h));
          sum[h] += z[h];
        }
      }

      // ---- P_b = p * s_b, a row's heads in one 128-byte row
      auto put = [&](float s, uint32_t group) {
        uint32_t u[HG / 2];
#pragma unroll
        for (int h = 0; h < HG / 2; ++h) {
          float lo, hi;
          mul2(lo, hi, s, z[2 * h], z[2 * h + 1]);
          u[h] = bf16x2(lo, hi);
        }
        uint8_t *at = sm + L::k + group * kGroupBytes + mine * 128;
        const uint32_t x = mine & 7;
#pragma unroll
        for (uint32_t c = 0; c < HG / 8; ++c)
          *reinterpret_cast<uint4 *>(at + (((HG / 8 * grp + c) ^ x) << 4)) = make_uint4(u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]);
      };
      put(scale.x, 8);
      hand_over(kBarP);
      Place next = w;
      step<NH>(p, next, words);
      if (more) fetch(raw2, n + 1, block2, 0);
      if (!(ok = warp_wait(bar(kBarPV), par))) break;
      put(scale.y, 0);
      put(scale.z, 8);
      put(scale.w, 1);
      hand_over(kBarP + 1);
      start = false;
      if (more) fetch(raw2, n + 1, block2, 1);

      // ---- the end of a piece: normalise and write (a warp's 32 lanes: 32 channels of a head)
      const bool item_ends = w.tile + 1 == p.tiles;
      if (item_ends || n + 1 == count) {
        const float mine_sum = sum_rows<HG>(sum, lane);
        if (lane < HG) top[lane * 4 + quad] = mine_sum;
        if (!(ok = exchange())) break;
        const float4 t4 = *reinterpret_cast<const float4 *>(top + (lane & (HG - 1)) * 4);
        const float total = (t4.x + t4.y) + (t4.z + t4.w), inv = total == 0.f ? 0.f : 1.f / total;
        const bool whole = !kCluster && item_ends && first_tile == 0;
        const uint32_t slot = 2 * blockIdx.x + (first_tile == 0 ? 1 : 0);
        if (quad == 0 && lane < HG) {
          const uint32_t head = grp * HG + lane;
          const float l2 = (ref == -INFINITY ? 0.f : ref) + log2f(total);
          if (kCluster)
            reinterpret_cast<float *>(sm + L::scale)[head] = l2;
          else if (!whole)
            p.part_lse[(uint64_t)slot * NH + head] = l2;
          else if (p.a.lse && w.h0 + head < p.a.heads)
            p.a.lse[(uint64_t)w.token * p.a.heads + w.h0 + head] = l2 * 0.693147180559945309f;
        }
#pragma unroll
        for (int h = 0; h < HG; ++h) sum[h] = __shfl_sync(0xffffffffu, inv, h);
        const uint32_t h0 = w.h0 + grp * HG;
        const int heads = p.a.heads < h0 ? 0 : p.a.heads - h0 < HG ? (int)(p.a.heads - h0) : HG;
        __nv_bfloat16 *out = (__nv_bfloat16 *)p.a.out + ((uint64_t)w.token * p.a.heads + h0) * ULA_ROW_LATENT + mine;
        float *part = p.part_out + ((uint64_t)slot * NH + grp * HG) * ULA_ROW_LATENT + mine;
        // (a cluster's results lie across the whole tile's room: no product may read it any more)
        if (kCluster && !(ok = warp_wait(bar(kBarPV + 3), par))) break;
#pragma unroll 1
        for (uint32_t b = 0; b < 4; ++b) {
          if (!(ok = warp_wait(bar(kBarPV + b), par))) break;
          tc_fence_after();
          float o[HG];
          tmem_ld<HG>(lanes + b * NH + grp * HG, o);
          tc_wait_ld();
          if (kCluster) {
            float *at = reinterpret_cast<float *>(sm + L::k) + grp * HG * ULA_ROW_LATENT + b * 128 + mine;
#pragma unroll
            for (int h = 0; h < HG; ++h) at[h * ULA_ROW_LATENT] = o[h] * sum[h];
          } else if (whole) {
#pragma unroll
            for (int h = 0; h < HG; ++h)
              if (h < heads) out[h * (int)ULA_ROW_LATENT + b * 128] = __float2bfloat16_rn(o[h] * sum[h]);
          } else {
#pragma unroll
            for (int h = 0; h < HG; ++h)
              if (h < heads) part[h * (int)ULA_ROW_LATENT + b * 128] = o[h] * sum[h];
          }
        }
        if (!ok) break;
        start = true;
      }
      w = next;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // (the queries of a warp that gave up before it used them)
    if (kCluster) {  // (here, since the other warps have fewer registers)
      tc_fence_before();
      meet();
      const uint32_t item = blockIdx.x / p.cluster, rank = blockIdx.x - item * p.cluster;
      const uint32_t token = item / p.head_tiles, h0 = (item - token * p.head_tiles) * NH;
      const uint32_t heads = p.a.heads - h0 < NH ? p.a.heads - h0 : NH;
      // this block's share: query heads [first, last).  The first values are on their way while
      // each part's weight in a head is worked out.
      const uint32_t first = rank * heads / p.cluster, last = (rank + 1) * heads / p.cluster;
      const uint32_t total = (last - first) * 128;
      float *weight = reinterpret_cast<float *>(sm + L::q);  // [head][part] (no product reads the queries any more)
      float4 o[kMostCluster];
      auto load = [&](uint32_t i) {
#pragma unroll
        for (uint32_t k = 0; k < kMostCluster; ++k)
          if (k < p.cluster) {
            uint32_t at;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(sk + first * 2048 + i * 16), "r"(k));
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(o[k].x), "=f"(o[k].y), "=f"(o[k].z), "=f"(o[k].w) : "r"(at) : "memory");
          }
      };
      uint32_t i = threadIdx.x;
      if (i < total) load(i);
      if (i < last - first) {
        const uint32_t h = first + i;
        float l[kMostCluster], m = -INFINITY, all = 0.f;
#pragma unroll
        for (uint32_t k = 0; k < kMostCluster; ++k) {
          l[k] = -INFINITY;
          if (k < p.cluster) {
            uint32_t at;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(base + L::scale + h * 4), "r"(k));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(l[k]) : "r"(at) : "memory");
          }
        }
#pragma unroll
        for (uint32_t k = 0; k < kMostCluster; ++k) m = fmaxf(m, l[k]);
        if (m == -INFINITY) m = 0.f;
#pragma unroll
        for (uint32_t k = 0; k < kMostCluster; ++k) all += l[k] = ex2(l[k] - m);
        const float inv = all == 0.f ? 0.f : 1.f / all;
#pragma unroll
        for (uint32_t k = 0; k < kMostCluster; ++k) weight[i * kMostCluster + k] = l[k] * inv;
        if (p.a.lse) p.a.lse[(uint64_t)token * p.a.heads + h0 + h] = (m + log2f(all)) * 0.693147180559945309f;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
      while (i < total) {
        const uint32_t h = i >> 7, c = i & 127;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (uint32_t k = 0; k < kMostCluster; ++k)
          if (k < p.cluster) {
            const float f = weight[h * kMostCluster + k];
            acc.x += f * o[k].x, acc.y += f * o[k].y, acc.z += f * o[k].z, acc.w += f * o[k].w;
          }
        reinterpret_cast<uint2 *>((__nv_bfloat16 *)p.a.out + ((uint64_t)token * p.a.heads + h0 + first + h) * ULA_ROW_LATENT)[c] =
            make_uint2(bf16x2(acc.x, acc.y), bf16x2(acc.z, acc.w));
        i += kWarps * 32;
        if (i < total) load(i);
      }
    }
  }
  if (!ok && lane == 0) atomicAdd(&g_late, 1u);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarps)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  // (a block's shared memory stays until the others have read it)
  if (kCluster) meet();
}

// Joins the partial results of the items that several blocks share: 128 threads per query
// token and head, 4 channels each; a block's `heads` heads (blockIdx.y) are of one item.
// Bound by the parts' bytes, which each SM reads from L2 at some 30 B a clock: 16.8 MB, 16 parts
// of 512 heads, 2 us and the loads' latency.
template <uint32_t kBatch>
__global__ void __launch_bounds__(256) k_join_parts(const __grid_constant__ AttendParams p, uint32_t nh, uint32_t heads) {
  const uint32_t item = p.rounds * p.blocks + blockIdx.x, c = threadIdx.x & 127;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (every block: the next kernel follows both)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t token = item / p.head_tiles, h0 = (item - token * p.head_tiles) * nh;
  const unsigned long long s = (unsigned long long)blockIdx.x * p.tiles;
  auto owner = [&](unsigned long long tile) -> uint32_t {  // (64-bit divisions only where they have to be)
    const unsigned long long x = (tile + 1) * p.sharers - 1;
    return (x | p.rest) >> 32 ? (uint32_t)(x / p.rest) : (uint32_t)x / (uint32_t)p.rest;
  };
  const uint32_t b0 = owner(s), b1 = owner(s + p.tiles - 1);
  if (b0 == b1) return;  // written whole
  uint32_t last = (blockIdx.y + 1) * heads;
  if (last > p.a.heads - h0) last = p.a.heads - h0;
  for (uint32_t h = blockIdx.y * heads + (threadIdx.x >> 7); h < last; h += 2) {
    Joined j;
    for (uint32_t b = b0; b <= b1; b += kBatch) {
      float l[kBatch];
      float4 o[kBatch];
#pragma unroll
      for (uint32_t k = 0; k < kBatch; ++k) {
        l[k] = -INFINITY, o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (b + k <= b1) {
          const uint64_t row = ((uint64_t)2 * (b + k) + (b + k == b0 ? 1 : 0)) * nh + h;
          l[k] = __ldcs(p.part_lse + row);
          o[k] = __ldcs(reinterpret_cast<const float4 *>(p.part_out + row * ULA_ROW_LATENT) + c);
        }
      }
      j.add(l, o);
    }
    j.write(p.a, (uint64_t)token * p.a.heads + h0 + h, c);
  }
}

bool aligned(const void *p, uint64_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

std::atomic<uint32_t> g_hold{kBars};

struct Plan {
  uint32_t sms, nh, head_tiles, tiles, keys, blocks, rounds, sharers, cluster;
  unsigned long long rest;
  bool parts;  // some item's tiles lie in several blocks that are no cluster
  uint64_t workspace;
};

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, uint32_t block, uint32_t smem, uint32_t cluster,
                   cudaStream_t st, Args... args) {
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster, at[1].val.clusterDim.y = 1, at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <uint32_t NH, bool kTree>
cudaError_t prepare_attend(bool cluster) {
  // (idempotent and cheap; a per-device flag would have to know about device resets)
  auto kernel = cluster ? k_attend<NH, true, kTree> : k_attend<NH, false, kTree>;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shared<NH>::bytes);
}

// For lists ("tokens": query tokens, or requests whose tree shares its list) of k entries and own rows
// behind them, and each list's columns (its query heads, or its nodes' query heads).
bool make_plan(uint64_t tokens, uint32_t heads, uint32_t k, uint32_t own, Plan *pl) {
  if (tokens > 0x7fffffffull || heads > 0x7fffffffu || k > 0x7fffffffu - kTile || own > 0x7fffffffu - kTile - k)
    return false;
  pl->keys = k + own;
  pl->tiles = pl->keys ? (pl->keys + kTile - 1) / kTile : 1;
  // Heads per item: the fewest that hold them all, up to 64 (TMEM's columns).  The rows are widened
  // once an item, so heads are not split further: 96 tokens x 2,051 rows, 64 heads, 71.6 us with 64
  // and 95.7 with 32.  Rounding 32 heads up to 64 costs 9.4 -> 11.7 us (one token, 256 rows), 16 up
  // to 32 63.7 -> 67.9 us (128 tokens, 2,048 rows).
  pl->nh = heads <= 16 ? 16 : heads <= 32 ? 32 : 64;
  pl->head_tiles = (heads + pl->nh - 1) / pl->nh;
  const uint64_t items = tokens * pl->head_tiles;
  if (items > 0x7fffffffull || tokens * heads > 0x7fffffffull) return false;
  const uint64_t total = items * pl->tiles;
  const int sms = sm_count();
  if (sms < 1 || total > (1ull << 48)) return false;
  pl->sms = (uint32_t)sms;
  // An item's tiles on a cluster, when there is one tile per block.  A cluster's join is shared
  // by its blocks alone, where the second kernel's is by all SMs: it takes blocks enough that the
  // trip of all partial results through L2 is what counts, and fewer blocks for its wider results
  // (us with clusters, without; heads, tiles, query tokens):
  //   32 heads  7 x 5: 10.9, 10.3    7 x 15: 11.4, 11.2    2 x 19: 10.6, 9.9    2 x 57: 11.0, 11.1
  //             4 x 28: 10.9, 11.9
  //   64 heads  4 x 1: 14.2, 12.7    4 x 28: 15.2, 15.1    8 x 14: 16.0, 15.6    2 x 76: 15.7, 17.3
  //   16 heads  8 x 15: 9.3, 10.1    2 x 57: 9.3, 10.1
  // Clusters of more than 2 cannot use every SM (a cluster lies within one group of SMs), and those
  // that find no place run behind the others: 32 heads 4 x 38: 20.4, 12.0.
  pl->cluster = 1;
  if (pl->tiles > 1 && pl->tiles <= (pl->nh == 64 ? kMostCluster / 2 : kMostCluster) &&
      total >= (unsigned)sms * 2 / 5 && total <= (unsigned)(pl->tiles == 2 ? sms : sms * 3 / 4)) {
    pl->cluster = pl->tiles;
    pl->blocks = (uint32_t)total, pl->rounds = 0, pl->rest = 0, pl->sharers = 1;
    pl->parts = false;
    pl->workspace = 0;
    return true;
  }
  pl->blocks = total == 0 ? 1 : total < (unsigned)sms ? (uint32_t)total : (uint32_t)sms;
  if (total / pl->blocks > 0x7fffffffull) return false;
  // Whole items first: their results need no join (192 items of 17 tiles: 120 us, with even shares
  // of all tiles 125).
  pl->rounds = (uint32_t)(items / pl->blocks);
  pl->rest = (items - (uint64_t)pl->rounds * pl->blocks) * pl->tiles;
  pl->sharers = pl->rest && pl->rest < pl->blocks ? (uint32_t)pl->rest : pl->blocks;
  pl->parts = pl->rest && pl->tiles > 1;
  pl->workspace = pl->parts ? (uint64_t)2 * pl->blocks * pl->nh * (ULA_ROW_LATENT + 1) * 4 : 0;
  return true;
}

template <uint32_t NH, bool kTree>
cudaError_t launch_attend(const AttendParams &p, cudaStream_t st) {
  const cudaError_t e = prepare_attend<NH, kTree>(p.cluster > 1);
  if (e != cudaSuccess) return e;
  return launch(p.cluster > 1 ? k_attend<NH, true, kTree> : k_attend<NH, false, kTree>, p.blocks, kThreads, Shared<NH>::bytes, p.cluster, st, p);
}

template <bool kTree>
cudaError_t launch_plan(const Plan &pl, AttendParams &p, cudaStream_t st) {
  p.rest = pl.rest, p.blocks = pl.blocks, p.rounds = pl.rounds, p.sharers = pl.sharers, p.tiles = pl.tiles, p.head_tiles = pl.head_tiles, p.keys = pl.keys;
  p.cluster = pl.cluster;
  p.hold = g_hold.load(std::memory_order_relaxed);
  p.c0 = p.a.softmax_scale * 1.44269504088896341f;
  p.part_out = (float *)p.a.workspace;
  p.part_lse = p.part_out + (uint64_t)2 * pl.blocks * pl.nh * ULA_ROW_LATENT;
  cudaError_t e = pl.nh == 16 ? launch_attend<16, kTree>(p, st) : pl.nh == 32 ? launch_attend<32, kTree>(p, st) : launch_attend<64, kTree>(p, st);
  if (e != cudaSuccess) return e;
  if (pl.parts) {
    // Heads per block of the join: 4 share the work on a block's place once every SM has several
    // blocks (96 tokens x 2,051 rows, 64 heads, both kernels: 72.9 us; 73.9 with 2), and 2 keep the
    // loads of few items on more SMs (8 tokens: 17.6 us; 21.2 with 4).
    // Parts in flight per thread: what an item can have up to 4 (one token, 2 parts: 9.4 us with
    // room for 2, 9.8 with 8; 96 tokens, 2 or 3: 72.9 us with 4, 76.3 with 8), else 16 while
    // there is a place for every block at that many registers (8 tokens, 16 parts: 15.6 us; 17.6
    // with 8), then 8 (20 tokens, 9 parts: 24.7 us; 26.7 with 16).
    const uint32_t items = (uint32_t)(pl.rest / pl.tiles), most = pl.sharers / items + 2;
    const uint32_t join_heads = (uint64_t)items * pl.nh / 4 >= 4ull * pl.sms ? 4 : 2;
    const bool few = (uint64_t)items * pl.nh / join_heads <= 2ull * pl.sms;
    e = launch(pl.tiles <= 2 ? k_join_parts<2> : pl.tiles <= 4 || most <= 4 ? k_join_parts<4> : few ? k_join_parts<16> : k_join_parts<8>,
               dim3(items, pl.nh / join_heads), 256, 0, 1, st, p, pl.nh, join_heads);
  }
  return e;
}

// What both calls ask of their arguments, whose strides along a single request, token or head count for
// nothing and become 0.
bool arguments_hold(ula_attend_args &a) {
  if (a.n_req == 1) a.q_req_stride = a.own_req_stride = 0;
  if (a.n_q == 1) a.q_tok_stride = a.own_tok_stride = 0;
  if (a.heads == 1) a.q_head_stride = 0;
  if (a.n_req == 0 || a.n_q == 0 || a.heads == 0) return true;
  if (!a.q || !a.out || (a.k && (!a.entry_row || (!a.rows && a.n_rows)))) return false;
  if (!aligned(a.q, 16) || !aligned(a.rows, 16) || !aligned(a.own_rows, 16) || !aligned(a.out, 16) ||
      !aligned(a.entry_row, 4) || !aligned(a.lse, 4) || !aligned(a.workspace, 16))
    return false;
  return !(a.q_req_stride % 8 || a.q_tok_stride % 8 || a.q_head_stride % 8 || a.own_req_stride % 16 ||
           a.own_tok_stride % 16 || a.n_rows > 0x7fffffffu);
}

}  // namespace

extern "C" uint64_t ula_rows_attend_workspace(uint32_t n_req, uint32_t n_q, uint32_t heads,
                                              uint32_t k, int own) {
  Plan pl;
  return make_plan((uint64_t)n_req * n_q, heads, k, own ? n_q : 0, &pl) ? pl.workspace : 0;
}

extern "C" int ula_rows_attend(const ula_attend_args *args, void *stream) {
  if (!args) return ULA_ERR_INVALID_ARG;
  AttendParams p{};
  p.a = *args;
  if (!arguments_hold(p.a)) return ULA_ERR_INVALID_ARG;
  if (p.a.n_req == 0 || p.a.n_q == 0 || p.a.heads == 0) return ULA_OK;
  Plan pl;
  if (!make_plan((uint64_t)p.a.n_req * p.a.n_q, p.a.heads, p.a.k, p.a.own_rows ? p.a.n_q : 0, &pl)) return ULA_ERR_INVALID_ARG;
  if (pl.workspace && (!p.a.workspace || p.a.workspace_bytes < pl.workspace)) return ULA_ERR_INVALID_ARG;
  return launch_plan<false>(pl, p, (cudaStream_t)stream) == cudaSuccess ? ULA_OK : ULA_ERR_CUDA;
}

namespace {

// The plan of a tree: lists of the nodes or, shared, of the requests.
bool plan_tree(uint32_t n_req, uint32_t n_q, uint32_t heads, uint32_t k, uint32_t flags, Plan *pl) {
  if (n_q > ULA_MAX_TREE || (flags & ~ULA_TREE_SHARED_LIST)) return false;
  const bool shared = flags & ULA_TREE_SHARED_LIST;
  if (shared && heads > 0x7fffffffu / ULA_MAX_TREE) return false;
  return make_plan(shared ? n_req : (uint64_t)n_req * n_q, shared ? n_q * heads : heads, k, n_q, pl);
}

}  // namespace

extern "C" uint64_t ula_rows_attend_tree_workspace(uint32_t n_req, uint32_t n_q, uint32_t heads, uint32_t k,
                                                   uint32_t flags) {
  Plan pl;
  return plan_tree(n_req, n_q, heads, k, flags, &pl) ? pl.workspace : 0;
}

extern "C" int ula_rows_attend_tree(const ula_attend_args *args, const int32_t *parent, uint32_t flags,
                                    void *stream) {
  if (!args) return ULA_ERR_INVALID_ARG;
  AttendParams p{};
  p.a = *args;
  if (!arguments_hold(p.a) || p.a.n_q > ULA_MAX_TREE || (flags & ~ULA_TREE_SHARED_LIST)) return ULA_ERR_INVALID_ARG;
  if (p.a.n_req == 0 || p.a.n_q == 0 || p.a.heads == 0) return ULA_OK;
  if (!p.a.own_rows || !parent || !aligned(parent, 4)) return ULA_ERR_INVALID_ARG;
  Plan pl;
  if (!plan_tree(p.a.n_req, p.a.n_q, p.a.heads, p.a.k, flags, &pl)) return ULA_ERR_INVALID_ARG;
  if (pl.workspace && (!p.a.workspace || p.a.workspace_bytes < pl.workspace)) return ULA_ERR_INVALID_ARG;
  p.parent = parent, p.nodes = p.a.n_q, p.node_heads = p.a.heads;
  if (flags & ULA_TREE_SHARED_LIST) p.a.heads *= p.a.n_q, p.a.n_q = 1;
  return launch_plan<true>(pl, p, (cudaStream_t)stream) == cudaSuccess ? ULA_OK : ULA_ERR_CUDA;
}

extern "C" int ula_rows_debug_hold(int barrier) {
  if (barrier >= (int)kBars) return ULA_ERR_INVALID_ARG;
  g_hold.store(barrier < 0 ? (uint32_t)kBars : (uint32_t)barrier, std::memory_order_relaxed);
  return ULA_OK;
}

// The count of late warps at each stream's last sync (0 where it stands at none).  Kept per stream,
// so that no stream's sync takes an error that another's results depend on.
extern "C" int ula_rows_sync(void *stream) {
  static std::mutex lock;
  static std::map<std::pair<int, unsigned long long>, uint32_t> seen;
  cudaStream_t st = (cudaStream_t)stream;
  uint32_t late = 0, late_scores = 0;
  int device = 0;
  unsigned long long id = 0;
  if (cudaMemcpyFromSymbolAsync(&late, g_late, sizeof late, 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      score_late(&late_scores, st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
    return ULA_ERR_CUDA;
  late += late_scores;
  if (late == 0) return ULA_OK;
  if (cudaGetDevice(&device) != cudaSuccess || cudaStreamGetId(st, &id) != cudaSuccess) return ULA_ERR_CUDA;
  try {
    const std::lock_guard<std::mutex> held(lock);
    uint32_t &last = seen[{device, id}];
    return std::exchange(last, late) == late ? ULA_OK : ULA_ERR_TIMEOUT;
  } catch (...) {  // (no memory for the entry: the error is returned, and again next time)
    return ULA_ERR_TIMEOUT;
  }
}
