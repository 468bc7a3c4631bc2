// Accumulated attention weights (ula_rows_score): scores[address[e]] += sum over the query heads that
// select e of exp(z[e] - lse), with the logits z of ula_rows_attend and the lse that it gave.
//
// An address may be selected by several query tokens, so its weights are summed as whole numbers, whose sum
// does not depend on their order; one addition in fp32 per address then updates its score.  A sum has two
// 64-bit words: units of 2^-e, with e such that no sum of this call's weights passes 2^62, and under them units
// of 2^-2e for what is left of a row's sum, which only a sum below 2^(24 - e) has (96 tokens, 2,048 rows, 128 heads:
// e = 37).  The first word's top bit says that there is a second, so that few are read: reading it for
// every entry took 66 us where this takes 55.5.  Three launches: the first clears the
// sums at the addresses in question and lays the queries out as the second reads them; the second adds
// the weights up; in the third each sum is taken by the first entry that finds it.
#include <cuda_bf16.h>
#include <atomic>
#include <cmath>

#include "ula.h"
#include "ula_tc.cuh"

using namespace ula_tc;

namespace {

constexpr unsigned long long kRest = 1ull << 63;  // (of a sum's first word)

struct ScoreParams {
  ula_score_args a;
  uint32_t lists, nodes;        // lists, and the query tokens of each
  ulonglong2 *sums;             // [n_scores]
  unsigned long long total;     // tiles of all items
  uint32_t tiles, column_tiles; // of an item; of a list
  uint8_t *images;              // [lists][column_tiles] the queries as they stand in shared memory
  uint32_t hold;                // (test hook) an mbarrier whose phases never end; kBars: none
  float c0, unit;               // softmax_scale * log2(e); 2^e
};

__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The queries of an item (a list's tile of NC columns): nine groups of 64 channels, [NC][128 B] each with
// the products' swizzle, then each column's -lse in units of log2 and the factor of its latents.
// A product's sum runs over channels in any order, so long as both sides have the same: that in which
// k_score's threads bring a row's 128 into TMEM.  Thread i of a row's four holds channels 16 i.. and 64 + 16 i..
// (of the rope channels 8 i.. and 32 + 8 i..), and gives 4 of them to every 16: the 16-byte chunk m
// holds the (m / 2)-th four channels of thread 2 (m % 2), then those of the next thread.
template <uint32_t NC>
struct Image {
  static constexpr uint32_t lse = 9 * NC * 128, factor = lse + NC * 4, bytes = factor + NC * 4;
};

// Clears the sums, and makes the images, a warp a column.  Bound by its bytes (a query is read and
// written once).  The latents become f16: exact once they are multiplied by a power of two that brings
// the column's largest near 2^15 (bf16 has 8 significant bits, and f16 keeps them down to 2^-31 of the
// largest; below, an error of 2^-39 of it is far under what fp32 sums lose).  The rope channels stay bf16.
template <uint32_t NC>
__global__ void __launch_bounds__(256) k_score_prepare(const __grid_constant__ ScoreParams p) {
  after_previous();
  const uint64_t n = (uint64_t)p.lists * p.a.k, stride = (uint64_t)gridDim.x * 256;
  uint64_t e = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  uint32_t a = e < n ? (uint32_t)__ldg(p.a.address + e) : 0xffffffffu;  // (on its way beside the first queries)
  const uint32_t lane = threadIdx.x & 31, columns = p.nodes * p.a.heads, per_list = p.column_tiles * NC;
  const uint64_t all = (uint64_t)p.lists * per_list;
  for (uint64_t i = (uint64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < all; i += (uint64_t)gridDim.x * 8) {
    const uint32_t list = (uint32_t)(i / per_list), c = (uint32_t)(i - (uint64_t)list * per_list), h = c % NC;
    uint8_t *image = p.images + (i / NC) * Image<NC>::bytes;
    uint8_t *dst = image + (lane >> 3) * (NC * 128) + h * 128 + (((lane & 7) ^ (h & 7)) << 4);
    // this lane's chunks, `lane` and `lane` + 32 of 64: chunk m of a block of 16
    const uint32_t m = lane & 15, j = m >> 1, at = (lane >> 4) * 128 + (j >> 2) * 64 + (m & 1) * 32 + (j & 3) * 4;
    const uint32_t at_rope = 512 + (lane >> 2) * 32 + (lane & 1) * 16 + (lane >> 1 & 1) * 4;
    uint4 v[2] = {}, rope = {};
    float l = -INFINITY;
    int up = 0;
    if (c < columns) {
      const uint32_t token = list * p.nodes + c / p.a.heads, head = c % p.a.heads, req = token / p.a.n_q;
      const __nv_bfloat16 *q = (const __nv_bfloat16 *)p.a.q + req * p.a.q_req_stride + (token - req * p.a.n_q) * p.a.q_tok_stride + head * p.a.q_head_stride;
      auto four = [&](uint32_t c4) { return __ldg(reinterpret_cast<const uint2 *>(q + c4)); };
      auto both = [&](uint32_t c4, uint32_t next) {
        const uint2 a = four(c4), b = four(c4 + next);
        return make_uint4(a.x, a.y, b.x, b.y);
      };
      v[0] = both(at, 16), v[1] = both(at + 256, 16);
      if (lane < 8) rope = both(at_rope, 8);
      l = __ldg(p.a.lse + (uint64_t)list * columns + c);
      uint32_t *u = reinterpret_cast<uint32_t *>(v), most = 0;  // the largest finite value's exponent
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t lo = u[k] >> 7 & 0xff, hi = u[k] >> 23 & 0xff;
        most = max(most, max(lo == 255 ? 0 : lo, hi == 255 ? 0 : hi));
      }
      most = __reduce_max_sync(0xffffffffu, most);
      up = min(14 + 127 - (int)most, 126);  // its exponent becomes 14; both factors are normal numbers of fp32
      const float by = __int_as_float((127 + up) << 23);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const __half2 t = __floats2half2_rn(__uint_as_float(u[k] << 16) * by, __uint_as_float(u[k] & 0xffff0000u) * by);
        u[k] = *reinterpret_cast<const uint32_t *>(&t);
      }
    }
    *reinterpret_cast<uint4 *>(dst) = v[0];
    *reinterpret_cast<uint4 *>(dst + 4 * NC * 128) = v[1];
    if (lane < 8) *reinterpret_cast<uint4 *>(dst + 8 * NC * 128) = rope;
    if (lane == 0) {  // (a column without an lse, or none: exp2(z - inf) is 0)
      reinterpret_cast<float *>(image + Image<NC>::lse)[h] = l > -INFINITY ? -l * 1.44269504088896341f : -INFINITY;
      reinterpret_cast<float *>(image + Image<NC>::factor)[h] = __int_as_float((127 - up) << 23);
    }
  }
  for (; e < n; e += stride) {
    if (a < p.a.n_scores) p.sums[a] = make_ulonglong2(0, 0);
    a = e + stride < n ? (uint32_t)__ldg(p.a.address + e + stride) : 0xffffffffu;
  }
}

// (Two calls that update the same scores at once: each adds its own sums.)  The addresses are read before the
// kernel before this one ends: it has waited for what came before it, so that nothing writes them any more.
__global__ void __launch_bounds__(256) k_score_commit(const __grid_constant__ ScoreParams p) {
  const uint64_t n = (uint64_t)p.lists * p.a.k, stride = (uint64_t)gridDim.x * 256;
  const double scale = 1.0 / (double)p.unit;
  uint64_t e = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  uint32_t a = e < n ? (uint32_t)__ldg(p.a.address + e) : 0xffffffffu;
  after_previous();
  for (; e < n; e += stride) {
    if (a < p.a.n_scores) {
      const unsigned long long s = atomicExch(&p.sums[a].x, 0ull);
      if (s) {
        double v = (double)(s & ~kRest) * scale;
        if (s & kRest) v += (double)__ldcg(&p.sums[a].y) * scale * scale;
        atomicAdd(p.a.scores + a, (float)v);
      }
    }
    a = e + stride < n ? (uint32_t)__ldg(p.a.address + e + stride) : 0xffffffffu;
  }
}

// ---------------------------------------------------------------- the weights

constexpr uint32_t kTile = 128;                      // rows per tile
constexpr uint32_t kPieces = 5;                      // of a tile: 4 blocks of latents, the rope channels
constexpr uint32_t kMostBufs = 4, kMostStages = 4;    // accumulators and pieces in TMEM
constexpr uint32_t kEnd = 8, kWiden = 8;             // warps that finish the logits, that widen rows
constexpr uint32_t kIssue = 2;                       // and that issue products; then one that looks rows up, one for the queries
constexpr uint32_t kThreads = (kEnd + kWiden + 4) * 32;  // (registers move between groups of 4 warps)
// Launched with 96 registers a thread: 5 * 96 = 2 * 128 + 2 * 80 + 64.
constexpr uint32_t kRegsEnd = 128, kRegsWiden = 80, kRegsIssue = 64;
constexpr uint32_t kParts = kEnd / 4;                // a row's columns are shared by so many threads
__device__ uint32_t g_late;                          // warps whose waits ran out, in all launches so far

// mbarriers.  Full, Empty: a stage holds a piece, its products have ended; Done, Drained: an
// accumulator stands, has been read; Place: the rows' addresses and targets stand; Scale: their scales;
// Free: all three have been read; Sum: the rows' sums stand; Query: the item's queries (of a piece's
// channels); Idle: the item's products with them have ended; End: an issuing warp's have.  (A wait names
// its phase by its parity alone, so whoever waits for a phase has to know that the one before it has ended: from
// a wait of its own or, for an issuing warp, which sees every other piece, from an accumulator that it has
// waited for, since those are read in the pieces' order and a product is issued after its queries stood.  The
// queries' last phase may be that of piece g - 5, so an accumulator of piece g - 5 or a later one has to have
// been read: the one that piece g - 2 waited for, where there are three, else the one that piece g waits for.)
constexpr uint32_t kTiles = 4;                       // tiles whose addresses, scales and sums stand at once
enum {
  kBarFull = 0, kBarEmpty = kBarFull + kMostStages, kBarDone = kBarEmpty + kMostStages, kBarDrained = kBarDone + kMostBufs,
  kBarPlace = kBarDrained + kMostBufs, kBarScale = kBarPlace + kTiles, kBarFree = kBarScale + kTiles,
  kBarSum = kBarFree + kTiles, kBarQuery = kBarSum + kTiles, kBarIdle = kBarQuery + kPieces, kBarEnd = kBarIdle + kPieces,
  kBars = kBarEnd + kIssue
};
static_assert(kBars == ULA_DEBUG_SCORE_BARRIERS, "as the header says");

template <uint32_t NC>
struct Shared {
  // TMEM: accumulators of NC columns, then stages of 64 (a piece of 128 channels)
  static constexpr uint32_t bufs = NC == 128 ? 3 : kMostBufs, stages = NC == 128 ? 2 : kMostStages;
  static_assert(bufs * NC + stages * 64 <= 512, "columns of TMEM");
  static constexpr uint32_t q = 0;                                  // [9][NC][128 B]
  static constexpr uint32_t scale = 9 * NC * 128;                   // [kTiles][128][4]
  static constexpr uint32_t place = scale + kTiles * kTile * 16;    // [kTiles][128] the rows' addresses (a query's: no row)
  static constexpr uint32_t target = place + kTiles * kTile * 8;    // [kTiles][128] their places in scores
  static constexpr uint32_t sum = target + kTiles * kTile * 4;      // [kTiles][kParts][128]
  static constexpr uint32_t lse = sum + kTiles * kParts * kTile * 4;     // [2][2][NC] -lse in units of log2, factors
  static constexpr uint32_t bars = lse + 4 * NC * 4;
  static constexpr uint32_t words = bars + kBars * 8;
  static constexpr uint32_t bytes = words + 16 + 1024;              // (+ alignment of the base)
};

// The tiles of a block: items (a list and a tile of its columns) in order, an even share of all tiles.
struct Place {
  uint32_t item, tile;
};

// S^T[128 rows][NC columns] = C_b Q_b^T for the four blocks of latents and the rope channels, as in the
// attention (ula_attend.cu), with the blocks' scales applied in fp32 as the accumulators are read.
// Codes are exact in f16, by one conversion for two of them.
// Nothing but the sum over a row's columns of exp2(z - lse) leaves the block, so the pieces of a
// tile stream: eight warps widen them into a ring of stages, two warps issue their products in turn into
// a ring of accumulators, eight warps take them up, a row per thread and half of the columns,
// and one adds the rows' sums to those in memory.
// The widened rows stand in TMEM, as the products' A: through shared memory a product of K = 16 read 8 KB of
// operands at what shared memory gives in all (118 B a clock), and every other access of the widening
// waited for it; now it reads the queries' 4 KB (96 tokens, 2,048 rows, 128 heads, the three kernels and
// a copy of the scores: 77 us before, 61 after).
//
// What bounds it: hand-overs.  A tile takes some 6,800 clocks (the case above: 40 us of 55, 0.73 PFLOP/s; 16
// requests of 16 tokens that share a list of 2,048 rows, 128 heads: 101 us in all, 0.76),
// its 36 products 2,300; the widening warps need 5,000 to 7,000 and the finishing ones 5,000, most of it in
// barriers that answer after 150 to 250 clocks.  (57 us when they were compared; 16 finishing warps of a quarter
// of the columns 62, for want of registers; 4 stages with 2 accumulators, or 3 with 2, the same within 1 %.)  Item tiles of up
// to 128 columns: the rows are widened once for all of them.
template <uint32_t NC>
__global__ void __launch_bounds__(kThreads, 1) k_score(const __grid_constant__ ScoreParams p) {
  extern __shared__ uint8_t raw_smem[];
  using L = Shared<NC>;
  constexpr uint32_t S = L::stages, kBufs = L::bufs;
  constexpr int HG = NC / kParts, kRead = HG < 32 ? HG : 32;  // columns of a thread, and of one read
  const uint32_t base = (smem_u32(raw_smem) + 1023u) & ~1023u;
  uint8_t *sm = raw_smem + (base - smem_u32(raw_smem));
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](uint32_t i) { return base + L::bars + 8 * i; };
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < kMostStages; ++i) mbar_init(bar(kBarFull + i), kWiden), mbar_init(bar(kBarEmpty + i), 1);
    for (uint32_t i = 0; i < kMostBufs; ++i) mbar_init(bar(kBarDone + i), 1), mbar_init(bar(kBarDrained + i), kEnd);
    for (uint32_t i = 0; i < kTiles; ++i) {
      mbar_init(bar(kBarPlace + i), 1), mbar_init(bar(kBarScale + i), 1);
      mbar_init(bar(kBarFree + i), kEnd + kWiden + 1), mbar_init(bar(kBarSum + i), kEnd);
    }
    for (uint32_t i = 0; i < kPieces; ++i) mbar_init(bar(kBarQuery + i), 1), mbar_init(bar(kBarIdle + i), 1);
    for (uint32_t i = 0; i < kIssue; ++i) mbar_init(bar(kBarEnd + i), 1);
    if (p.hold < kBars) {
      asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar(p.hold)) : "memory");
      mbar_init(bar(p.hold), 1u << 19);  // (more arrivals than a launch makes)
    }
    fence_async_smem();
  }
  // (An entry without a row stands for 656 bytes of the queries, whose products nobody adds up.  So does what
  // is read before its time, after a wait that ran out.)
  for (uint32_t i = threadIdx.x; i < kTiles * kTile; i += kThreads) {
    reinterpret_cast<uint64_t *>(sm + L::place)[i] = (uint64_t)p.a.q;
    reinterpret_cast<uint32_t *>(sm + L::target)[i] = 0xffffffffu;
  }
  if (warp == kEnd + kWiden) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + L::words) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm + L::words);
  const unsigned long long from = p.total * blockIdx.x / gridDim.x;
  const uint32_t count = (uint32_t)(p.total * (blockIdx.x + 1) / gridDim.x - from);
  Place w;
  w.item = (uint32_t)(from / p.tiles), w.tile = (uint32_t)(from - (unsigned long long)w.item * p.tiles);
  auto step = [&]() {
    if (++w.tile == p.tiles) w.tile = 0, ++w.item;
  };
  // The kernel before this one (k_score_prepare) has waited for all before it, so the rows, entries and
  // addresses stand; who touches the sums and the images waits for it, and so does every warp before it waits
  // for what depends on them: the limit of those waits is this kernel's alone.
  auto prepared = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
  if (warp == kEnd + kWiden + kIssue + 1) after_previous();

  bool ok = true;  // false once a wait has run out
  if (warp < kEnd) {
    // ---- logits, weights, sums: this thread's row and HG columns.  Whether the next accumulator stands is
    // asked before this one's numbers are added up.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEnd));
    const uint32_t quad = warp & 3, grp = warp >> 2, mine = 32 * quad + lane;
    const uint32_t lanes = tmem + (quad << 21) + grp * HG;
    uint32_t items = 0, stands = 0;
    prepared();
    for (uint32_t n = 0; n < count; ++n, step()) {
      const uint32_t at = n % kTiles, par = n / kTiles & 1;
      if (n == 0 || w.tile == 0) {  // (the lse come with the rope channels)
        if (!(ok = warp_wait(bar(kBarQuery + 4), items & 1))) break;
        ++items;
      }
      if (!(ok = warp_wait(bar(kBarScale + at), par))) break;
      const float4 s4 = *reinterpret_cast<const float4 *>(sm + L::scale + (at * kTile + mine) * 16);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarFree + at));
      float z[HG];
#pragma unroll
      for (uint32_t b = 0; b < kPieces; ++b) {
        const uint32_t g = n * kPieces + b, buf = g % kBufs;
        if (!__all_sync(0xffffffffu, stands) && !(ok = warp_wait(bar(kBarDone + buf), (g / kBufs) & 1))) break;
        tc_fence_after();
        float x[kRead];
        tmem_ld<kRead>(lanes + buf * NC, x);
        stands = mbar_ended(bar(kBarDone + (g + 1) % kBufs), ((g + 1) / kBufs) & 1);
        if (b == 4) {  // the latents' part as it was before its column was scaled, less the lse
          const float *l = reinterpret_cast<const float *>(sm + L::lse) + ((items - 1) & 1) * 2 * NC + grp * HG;
#pragma unroll
          for (int c = 0; c < HG; c += 4) {
            const float4 l4 = *reinterpret_cast<const float4 *>(l + c), f4 = *reinterpret_cast<const float4 *>(l + NC + c);
            fma2(z[c], z[c + 1], f4.x, f4.y, l4.x, l4.y);
            fma2(z[c + 2], z[c + 3], f4.z, f4.w, l4.z, l4.w);
          }
        }
        const float s = (b == 0 ? s4.x : b == 1 ? s4.y : b == 2 ? s4.z : b == 3 ? s4.w : 1.f) * p.c0;
#pragma unroll
        for (int c = 0; c < HG; c += kRead) {
          if (c) tmem_ld<kRead>(lanes + buf * NC + c, x);
          tc_wait_ld();
          if (c + kRead == HG) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarDrained + buf));
          }
#pragma unroll
          for (int h = 0; h < kRead; h += 2) {
            if (b == 0) mul2(z[c + h], z[c + h + 1], s, x[h], x[h + 1]);
            else fma2(z[c + h], z[c + h + 1], s, x[h], x[h + 1]);
          }
        }
      }
      if (!ok) break;
      // a weight is between 0 and 1, and 0 where it is not a number (what .sat makes of one)
      float total[4] = {};
#pragma unroll
      for (int c = 0; c < HG; c += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) total[i] += __saturatef(ex2(z[c + i]));
      reinterpret_cast<float *>(sm + L::sum)[(at * kParts + grp) * kTile + mine] = (total[0] + total[1]) + (total[2] + total[3]);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarSum + at));
    }
  } else if (warp < kEnd + kWiden) {
    // ---- widening: a warp 16 rows of every piece (half of its 32 lanes of TMEM); four lanes share a row
    // and hold another one 8 rows on, 32 bytes of each row's 128.  The loads of the next two pieces are in flight.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWiden));
    const uint32_t cw = warp - kEnd, first = 32 * (cw & 3) + 16 * (cw >> 2), r0 = first + (lane >> 2), ch = lane & 3;
    const uint32_t mine = tmem + kBufs * NC + (first << 16);
    const uint32_t pieces = count * kPieces;
    uint64_t row[2] = {};  // the rows of the tile whose pieces are being loaded
    auto fetch = [&](uint4 (&raw)[4], uint32_t g) -> bool {
      const uint32_t n = g / kPieces, b = g - n * kPieces;
      if (b == 0) {
        const uint32_t at = n % kTiles;
        if (!warp_wait(bar(kBarPlace + at), n / kTiles & 1)) return false;
        const uint64_t *place = reinterpret_cast<const uint64_t *>(sm + L::place) + at * kTile + r0;
        row[0] = place[0] + ch * 16, row[1] = place[8] + ch * 16;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarFree + at));
      }
      const uint32_t at = b < 4 ? b * 128 : ULA_ROW_LATENT + 16;
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) raw[j] = __ldg(reinterpret_cast<const uint4 *>(row[j >> 1] + at + (j & 1) * 64));
      return true;
    };
    uint32_t empty = 0;  // whether the next piece's stage is
    auto piece = [&](uint4 (&raw)[4], uint32_t g) -> bool {
      const uint32_t b = g % kPieces, st = g % S;
      if (g >= S && !__all_sync(0xffffffffu, empty) && (prepared(), !warp_wait(bar(kBarEmpty + st), (g / S & 1) ^ 1))) return false;
      tc_fence_after();
      const uint32_t stage = mine + st * 64;
      if (b == 4) {
        const uint32_t v[16] = {raw[0].x, raw[0].y, raw[2].x, raw[2].y, raw[0].z, raw[0].w, raw[2].z, raw[2].w,
                                raw[1].x, raw[1].y, raw[3].x, raw[3].y, raw[1].z, raw[1].w, raw[3].z, raw[3].w};
        tmem_st_16x32(stage, v);
      } else {
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i) {
          const uint4 a = raw[i], c = raw[2 + i];  // 16 codes of the first row, of the second
          const uint32_t v[16] = {codes_to_f16(a.x), codes_to_f16(a.x >> 16), codes_to_f16(c.x), codes_to_f16(c.x >> 16),
                                  codes_to_f16(a.y), codes_to_f16(a.y >> 16), codes_to_f16(c.y), codes_to_f16(c.y >> 16),
                                  codes_to_f16(a.z), codes_to_f16(a.z >> 16), codes_to_f16(c.z), codes_to_f16(c.z >> 16),
                                  codes_to_f16(a.w), codes_to_f16(a.w >> 16), codes_to_f16(c.w), codes_to_f16(c.w >> 16)};
          tmem_st_16x32(stage + 32 * i, v);
        }
      }
      empty = mbar_ended(bar(kBarEmpty + (g + 1) % S), ((g + 1) / S & 1) ^ 1);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarFull + st));
      return g + 2 >= pieces || fetch(raw, g + 2);
    };
    uint4 raw0[4], raw1[4];
    ok = pieces == 0 || (fetch(raw0, 0) && fetch(raw1, 1));  // (a tile has five)
    for (uint32_t g = 0; g < pieces && ok; g += 2) ok = piece(raw0, g) && (g + 1 >= pieces || piece(raw1, g + 1));
  } else if (warp < kEnd + kWiden + kIssue) {
    // ---- products, every other piece.  (A wait that has run out does not leave the loop, so that the
    // descriptors stay in uniform registers; it is reported at the end.)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    const uint32_t which = warp - kEnd - kWiden;
    // D fp32; A and B f16, the rope channels bf16
    constexpr uint32_t kId = (1u << 4) | ((NC >> 3) << 17) | ((kTile >> 4) << 24), kIdRope = kId | (1u << 7) | (1u << 10);
    const uint64_t queries = operand(base + L::q, 16);
    uint32_t items = 0, tile = 0;
    const uint32_t pieces = count * kPieces;
    prepared();
    for (uint32_t g = which; g < pieces; g += kIssue) {
      const uint32_t n = g / kPieces, b = g - n * kPieces, st = g % S, buf = g % kBufs;
      for (; tile < n; ++tile) step();
      if (n == 0 || w.tile == 0) {
        static_assert(kBufs <= kPieces, "an accumulator's wait tells that an earlier item's queries stood");
        if (kBufs + kIssue > kPieces && g >= kBufs) ok = ok && warp_wait(bar(kBarDrained + buf), (g / kBufs & 1) ^ 1);
        if (b < 2) ++items;
        ok = ok && warp_wait(bar(kBarQuery + b), (items - 1) & 1);
      }
      const uint32_t ready = g >= kBufs ? mbar_ended(bar(kBarFull + st), (g / S) & 1, bar(kBarDrained + buf), (g / kBufs & 1) ^ 1) : 0;
      if (!__all_sync(0xffffffffu, ready)) {
        ok = ok && warp_wait(bar(kBarFull + st), (g / S) & 1);
        if (g >= kBufs) ok = ok && warp_wait(bar(kBarDrained + buf), (g / kBufs & 1) ^ 1);
      }
      tc_fence_after();
      const uint64_t db = queries + b * (2 * NC * 128 >> 4);
      const uint32_t a = tmem + kBufs * NC + st * 64;
      if (elect_one()) {
#pragma unroll
        for (uint32_t s = 0; s < 8; ++s)
          if (s < 4 || b < 4)
            mma_tmem_a(tmem + buf * NC, a + 8 * s, db + (s >> 2) * (NC * 128 >> 4) + (s & 3) * 2, b < 4 ? kId : kIdRope, s != 0);
        mma_commit(bar(kBarEmpty + st));
        mma_commit(bar(kBarDone + buf));
        if (w.tile + 1 == p.tiles) mma_commit(bar(kBarIdle + b));
      }
      __syncwarp();
    }
    bool ended = true;
    if (elect_one()) {  // every product has ended before the block's TMEM goes
      mma_commit(bar(kBarEnd + which));
      ended = mbar_wait(bar(kBarEnd + which), 0);
    }
    ok = __all_sync(0xffffffffu, ended) && ok;
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
  }
  if (warp == kEnd + kWiden + kIssue) {
    // ---- the rows' addresses and targets, a tile ahead (four a lane), their scales, and the rows into L2
    int32_t u[4], to[4];
    auto fetch = [&]() {
      const uint32_t list = w.item / p.column_tiles;
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) {
        const uint32_t e = w.tile * kTile + lane + 32 * j;
        u[j] = to[j] = -1;
        if (e < p.a.k) {
          u[j] = __ldg(p.a.entry_row + (uint64_t)list * p.a.k + e);
          to[j] = __ldg(p.a.address + (uint64_t)list * p.a.k + e);
        }
      }
    };
    // (a tile's scales are stored when the next one's rows are known: waiting for them here made this warp the
    // slowest, 5,000 clocks a tile)
    float4 scale[4];
    auto store_scales = [&](uint32_t n) {
      float4 *to4 = reinterpret_cast<float4 *>(sm + L::scale) + n % kTiles * kTile + lane;
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) to4[32 * j] = scale[j];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarScale + n % kTiles));
    };
    if (count) fetch();
    for (uint32_t n = 0; n < count; ++n) {
      const uint32_t at = n % kTiles;
      if (n >= kTiles && (prepared(), !(ok = warp_wait(bar(kBarFree + at), (n / kTiles & 1) ^ 1)))) break;
      uint64_t row[4];
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) {
        const bool in = (uint32_t)u[j] < p.a.n_rows && (uint32_t)to[j] < p.a.n_scores;
        row[j] = in ? (uint64_t)p.a.rows + (uint64_t)(uint32_t)u[j] * ULA_ROW_BYTES : (uint64_t)p.a.q;
        reinterpret_cast<uint64_t *>(sm + L::place)[at * kTile + lane + 32 * j] = row[j];
        reinterpret_cast<uint32_t *>(sm + L::target)[at * kTile + lane + 32 * j] = in ? (uint32_t)to[j] : 0xffffffffu;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarPlace + at));
      if (n) store_scales(n - 1);
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) scale[j] = __ldg(reinterpret_cast<const float4 *>(row[j] + ULA_ROW_LATENT));
      step();
      if (n + 1 < count) fetch();
      if (n) {  // into L2 ahead of the loads, by lines: a bulk prefetch of a row takes its engine 64 clocks
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
#pragma unroll
          for (uint32_t i = 0; i < ULA_ROW_BYTES; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(row[j] + i));
      }
    }
    if (count && ok) store_scales(count - 1);
  }
  if (warp == kEnd + kWiden + kIssue + 1) {
    // ---- an item's queries, once the products that read the last one's have ended; a tile's sums, as whole
    // numbers, to those in memory (four rows a lane)
    uint32_t items = 0, begun = 0;  // items, and copies of pieces, begun
    auto load_queries = [&](uint32_t item) -> bool {  // piece by piece, as the last item's are done with
      for (uint32_t b = 0; b < kPieces; ++b, ++begun) {
        if (items && !(warp_wait(bar(kBarIdle + b), (items - 1) & 1) && warp_wait(bar(kBarQuery + b), (items - 1) & 1))) return false;
        if (elect_one()) {
          const uint8_t *image = p.images + (uint64_t)item * Image<NC>::bytes + b * 2 * NC * 128;
          const uint32_t bytes = b < 4 ? 2 * NC * 128 : NC * 128, more = b < 4 ? 0 : 2 * NC * 4, to = bar(kBarQuery + b);
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(to), "r"(bytes + more) : "memory");
          copy_bulk(base + L::q + b * 2 * NC * 128, image, bytes, to);
          if (more) copy_bulk(base + L::lse + (items & 1) * 2 * NC * 4, image + bytes, more, to);
        }
        __syncwarp();
      }
      ++items;
      return true;
    };
    if (count) ok = load_queries(w.item);
    for (uint32_t n = 0; n < count; ++n) {
      const uint32_t at = n % kTiles;
      step();
      if (w.tile == 0 && n + 1 < count && !(ok = load_queries(w.item))) break;
      if (!(ok = warp_wait(bar(kBarSum + at), n / kTiles & 1))) break;
      const float *sum = reinterpret_cast<const float *>(sm + L::sum) + at * kParts * kTile + lane;
      const uint32_t *target = reinterpret_cast<const uint32_t *>(sm + L::target) + at * kTile + lane;
#pragma unroll
      for (uint32_t j = 0; j < kTile; j += 32) {
        float total = 0.f;
#pragma unroll
        for (uint32_t i = 0; i < kParts; ++i) total += sum[i * kTile + j];
        if (target[j] != 0xffffffffu && total > 0.f) {
          ulonglong2 *to = p.sums + target[j];
          const float t = total * p.unit, whole = floorf(t), rest = t - whole;  // (all exact)
          atomicAdd(&to->x, __float2ull_rn(whole));
          if (rest > 0.f) {
            atomicAdd(&to->y, __float2ull_rn(rest * p.unit));
            atomicOr(&to->x, kRest);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarFree + at));
    }
    for (uint32_t b = 0; b < kPieces; ++b) {  // (no copy is in flight when the block ends)
      const uint32_t copies = begun / kPieces + (begun % kPieces > b ? 1 : 0);
      if (copies) ok = warp_wait(bar(kBarQuery + b), (copies - 1) & 1) && ok;
    }
  }
  if (!ok && lane == 0) atomicAdd(&g_late, 1u);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kEnd + kWiden)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

bool aligned(const void *p, uint64_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

cudaError_t launch(void (*kernel)(ScoreParams), uint64_t grid, uint32_t threads, uint32_t smem, cudaStream_t st, const ScoreParams &p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

std::atomic<uint32_t> g_hold{kBars};

int sm_count() {
  int dev = 0, n = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? n : 0;
}

template <uint32_t NC>
cudaError_t launch_score(ScoreParams &p, cudaStream_t st) {
  const uint32_t columns = p.nodes * p.a.heads;
  const int sms = sm_count();
  p.column_tiles = (columns + NC - 1) / NC;
  p.tiles = (p.a.k + kTile - 1) / kTile;
  p.total = (unsigned long long)p.lists * p.column_tiles * p.tiles;
  if (sms < 1) return cudaErrorInvalidDevice;
  // (idempotent and cheap; a per-device flag would have to know about device resets)
  cudaError_t e = cudaFuncSetAttribute(k_score<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shared<NC>::bytes);
  if (e != cudaSuccess) return e;
  const uint64_t warps = (uint64_t)p.lists * p.column_tiles * NC, entries = (uint64_t)p.lists * p.a.k;
  const uint64_t blocks = (warps + 7) / 8 > (entries + 255) / 256 ? (warps + 7) / 8 : (entries + 255) / 256;
  e = launch(k_score_prepare<NC>, blocks < 2048 ? blocks : 2048, 256, 0, st, p);
  if (e != cudaSuccess) return e;
  return launch(k_score<NC>, p.total < (unsigned)sms ? p.total : (unsigned)sms, kThreads, Shared<NC>::bytes, st, p);
}

}  // namespace

cudaError_t ula_tc::score_late(uint32_t *late, cudaStream_t st) {
  return cudaMemcpyFromSymbolAsync(late, g_late, sizeof *late, 0, cudaMemcpyDeviceToHost, st);
}

extern "C" int ula_rows_debug_hold_score(int barrier) {
  if (barrier >= (int)kBars) return ULA_ERR_INVALID_ARG;
  g_hold.store(barrier < 0 ? (uint32_t)kBars : (uint32_t)barrier, std::memory_order_relaxed);
  return ULA_OK;
}

namespace {

// Columns of an item: the fewest that hold a list's, up to 128 (TMEM's four accumulators).
uint32_t item_columns(uint64_t columns) { return columns <= 32 ? 32 : columns <= 64 ? 64 : 128; }
uint32_t image_bytes(uint32_t nc) { return nc == 32 ? Image<32>::bytes : nc == 64 ? Image<64>::bytes : Image<128>::bytes; }
uint64_t sums_bytes(uint32_t n_scores) { return ((uint64_t)n_scores * sizeof(ulonglong2) + 127) & ~127ull; }

}  // namespace

extern "C" uint64_t ula_rows_score_workspace(uint32_t n_req, uint32_t n_q, uint32_t heads, uint32_t flags, uint32_t n_scores) {
  const bool shared = flags & ULA_TREE_SHARED_LIST;
  const uint64_t lists = shared ? n_req : (uint64_t)n_req * n_q, columns = shared ? (uint64_t)n_q * heads : heads;
  const uint32_t nc = item_columns(columns);
  return sums_bytes(n_scores) + lists * ((columns + nc - 1) / nc) * image_bytes(nc);
}

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
      !aligned(a.lse, 4) || !aligned(a.scores, 4) || !aligned(a.workspace, 16) || a.q_req_stride % 8 ||
      a.q_tok_stride % 8 || a.q_head_stride % 8 || a.n_rows > 0x7fffffffu || a.n_scores > 0x7fffffffu ||
      a.workspace_bytes < ula_rows_score_workspace(a.n_req, a.n_q, a.heads, a.flags, a.n_scores))
    return ULA_ERR_INVALID_ARG;
  const bool shared = a.flags & ULA_TREE_SHARED_LIST;
  const uint64_t tokens = (uint64_t)a.n_req * a.n_q;
  p.nodes = shared ? a.n_q : 1;
  if (tokens > 0x7fffffffull || a.heads > 0x7fffffffu || tokens * a.heads > 0x7fffffffull || a.k > 0x7fffffffu ||
      (tokens * a.heads / 16 + tokens) * (a.k / 128 + 1ull) > (1ull << 36))
    return ULA_ERR_INVALID_ARG;
  p.lists = shared ? a.n_req : (uint32_t)tokens;
  p.sums = (ulonglong2 *)a.workspace;
  p.images = (uint8_t *)a.workspace + sums_bytes(a.n_scores);
  p.c0 = a.softmax_scale * 1.44269504088896341f;
  // a weight is at most 1, and an address gets at most one of every entry of every query head (and, a row at a
  // time, as many rests, each of 2^e at most)
  int bits = 2;
  while (tokens * a.heads * a.k > 1ull << bits) ++bits;
  p.unit = std::ldexp(1.f, 62 - bits);
  p.hold = g_hold.load(std::memory_order_relaxed);
  const uint64_t n = (uint64_t)p.lists * a.k, columns = (uint64_t)p.nodes * a.heads;
  cudaStream_t st = (cudaStream_t)stream;
  const uint64_t blocks = (n + 255) / 256 < 1024 ? (n + 255) / 256 : 1024;
  cudaError_t e = item_columns(columns) == 32 ? launch_score<32>(p, st) : item_columns(columns) == 64 ? launch_score<64>(p, st) : launch_score<128>(p, st);
  if (e == cudaSuccess) e = launch(k_score_commit, blocks, 256, 0, st, p);
  return e == cudaSuccess ? ULA_OK : ULA_ERR_CUDA;
}
